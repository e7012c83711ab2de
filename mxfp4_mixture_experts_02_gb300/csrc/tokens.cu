// Tokens into expert order and back, with their gradients.  c_map [T, k']
// holds the row of each slot (-1: the slot's expert is not here), so every
// direction is a walk over tokens with no atomics and a fixed order of sums:
//   permute            rows[c_map[t, j]] = x[t]
//   unpermute          out[t] = sum_j w[t, j] rows[c_map[t, j]]
//   permute's gradient is unpermute with weight 1, and
//   unpermute's        drows[c_map[t, j]] = w[t, j] dout[t],
//                      dw[t, j] = <dout[t], rows[c_map[t, j]]>, 0 at -1
// (the shapes of "[SGLang] CUTLASS MoE", sections 2 and 5, in the rows' own
// type).  Sums are in 32 bits, j ascending.
#include "train.cuh"

namespace moe {

namespace {

constexpr int kTokThreads = 128;
constexpr int kMaxSlots = 33;  // top_k <= 32 and one shared expert

// The token's map entries into shared memory.
__device__ __forceinline__ void load_slots(const TokenParams& p, int64_t t, int* s_row) {
    if (threadIdx.x < p.kp) s_row[threadIdx.x] = p.c_map[t * p.kp + threadIdx.x];
    __syncthreads();
}

// CTA (chunk of columns, token): the chunk is read once and written to the
// token's rows.
template <typename T, int VE>
__global__ void __launch_bounds__(kTokThreads) permute_kernel(TokenParams p) {
    __shared__ int s_row[kMaxSlots];
    ptx::pdl_wait();
    const int64_t t = blockIdx.x;
    load_slots(p, t, s_row);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kTokThreads + threadIdx.x) * VE;
    if (c >= p.H) return;
    const Vec<T, VE> v = load_vec<T, VE>(static_cast<const T*>(p.src) + t * p.H + c);
    for (int j = 0; j < p.kp; ++j) {
        const int64_t r = s_row[j];
        if (r >= 0) store_vec<T, VE>(static_cast<T*>(p.dst) + r * p.H + c, v);
    }
}

constexpr int kRowBatch = 4;  // rows in flight per thread

template <typename T, int VE>
__global__ void __launch_bounds__(kTokThreads) unpermute_kernel(TokenParams p) {
    __shared__ int s_row[kMaxSlots];
    __shared__ float s_w[kMaxSlots];
    const int64_t t = blockIdx.x;
    if (threadIdx.x < p.kp) s_w[threadIdx.x] = p.w ? p.w[t * p.kp + threadIdx.x] : 1.f;
    load_slots(p, t, s_row);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kTokThreads + threadIdx.x) * VE;
    if (c >= p.H) return;
    float acc[VE];
#pragma unroll
    for (int u = 0; u < VE; ++u) acc[u] = 0.f;
    for (int j0 = 0; j0 < p.kp; j0 += kRowBatch) {
        Vec<T, VE> v[kRowBatch];
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b) {
            const int64_t r = j0 + b < p.kp ? s_row[j0 + b] : -1;
            if (r >= 0) v[b] = load_vec<T, VE>(static_cast<const T*>(p.src) + r * p.H + c);
        }
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b) {
            if (j0 + b >= p.kp || s_row[j0 + b] < 0) continue;  // a slot without a row adds nothing
#pragma unroll
            for (int u = 0; u < VE; ++u) acc[u] += s_w[j0 + b] * to_f32(v[b].v[u]);
        }
    }
    Vec<T, VE> o;
#pragma unroll
    for (int u = 0; u < VE; ++u) o.v[u] = from_f32<T>(acc[u]);
    store_vec<T, VE>(static_cast<T*>(p.dst) + t * p.H + c, o);
}

constexpr int kGradTokThreads = 256;

// One CTA per token (a routing weight's gradient is a sum over the whole
// row): the warps' partial products gather in shared memory.
template <typename T, int VE>
__global__ void __launch_bounds__(kGradTokThreads) unpermute_grad_kernel(TokenParams p) {
    constexpr int kWarps = kGradTokThreads / 32;
    __shared__ int s_row[kMaxSlots];
    __shared__ float s_w[kMaxSlots];
    __shared__ float s_dot[kMaxSlots][kWarps];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < p.kp) s_w[threadIdx.x] = p.w[t * p.kp + threadIdx.x];
    for (int i = threadIdx.x; i < kMaxSlots * kWarps; i += kGradTokThreads) s_dot[i / kWarps][i % kWarps] = 0.f;
    load_slots(p, t, s_row);
    for (int64_t c0 = 0; c0 < p.H; c0 += kGradTokThreads * VE) {
        const int64_t c = c0 + threadIdx.x * VE;
        const bool in = c < p.H;
        float d[VE];
#pragma unroll
        for (int u = 0; u < VE; ++u) d[u] = 0.f;
        if (in) {
            const Vec<T, VE> v = load_vec<T, VE>(static_cast<const T*>(p.dout) + t * p.H + c);
#pragma unroll
            for (int u = 0; u < VE; ++u) d[u] = to_f32(v.v[u]);
        }
        for (int j0 = 0; j0 < p.kp; j0 += kRowBatch) {
            Vec<T, VE> y[kRowBatch];
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) {
                const int64_t r = j0 + b < p.kp ? s_row[j0 + b] : -1;
                if (in && r >= 0) y[b] = load_vec<T, VE>(static_cast<const T*>(p.src) + r * p.H + c);
            }
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) {
                const int64_t r = j0 + b < p.kp ? s_row[j0 + b] : -1;
                if (r < 0) continue;  // the same for the whole CTA
                float dot = 0.f;
                if (in) {
                    Vec<T, VE> o;
                    const float w = s_w[j0 + b];
#pragma unroll
                    for (int u = 0; u < VE; ++u) {
                        dot += d[u] * to_f32(y[b].v[u]);
                        o.v[u] = from_f32<T>(w * d[u]);
                    }
                    store_vec<T, VE>(static_cast<T*>(p.dst) + r * p.H + c, o);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (lane == 0) s_dot[j0 + b][warp] += dot;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x < p.kp) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += s_dot[threadIdx.x][i];
        p.dw[t * p.kp + threadIdx.x] = s;
    }
}

template <typename F>
cudaError_t by_type(int dtype, bool vec, F f) {
    switch (dtype) {
        case MOE_DTYPE_BF16:
            return vec ? f(__nv_bfloat16{}, std::integral_constant<int, 8>{})
                       : f(__nv_bfloat16{}, std::integral_constant<int, 1>{});
        case MOE_DTYPE_F16:
            return vec ? f(__half{}, std::integral_constant<int, 8>{}) : f(__half{}, std::integral_constant<int, 1>{});
        default:
            return vec ? f(float{}, std::integral_constant<int, 4>{}) : f(float{}, std::integral_constant<int, 1>{});
    }
}

dim3 token_grid(const TokenParams& p, int ve) {
    const int per = kTokThreads * ve;
    return dim3(p.T, (p.H + per - 1) / per);
}

}  // namespace

cudaError_t launch_permute(const TokenParams& p, int dtype, bool vec, cudaStream_t st, bool pdl) {
    return by_type(dtype, vec, [&](auto t, auto ve) {
        return launch_kernel(permute_kernel<decltype(t), ve.value>, token_grid(p, ve.value), dim3(kTokThreads), 0, st,
                             pdl, p);
    });
}

cudaError_t launch_unpermute(const TokenParams& p, int dtype, bool vec, cudaStream_t st) {
    return by_type(dtype, vec, [&](auto t, auto ve) {
        return launch_kernel(unpermute_kernel<decltype(t), ve.value>, token_grid(p, ve.value), dim3(kTokThreads), 0,
                             st, false, p);
    });
}

cudaError_t launch_unpermute_grad(const TokenParams& p, int dtype, bool vec, cudaStream_t st) {
    return by_type(dtype, vec, [&](auto t, auto ve) {
        return launch_kernel(unpermute_grad_kernel<decltype(t), ve.value>, dim3(p.T), dim3(kGradTokThreads), 0, st,
                             false, p);
    });
}

}  // namespace moe
