// Tokens into expert order and back, with their gradients.  c_map [T, k']
// holds the row of each slot (-1: the slot's expert is not here), so every
// direction is a walk over tokens with no atomics and a fixed order of sums:
//   permute            rows[c_map[t, j]] = x[t]
//   unpermute          out[t] = sum_j w[t, j] rows[c_map[t, j]]
//   permute's gradient is unpermute with weight 1, and
//   unpermute's        drows[c_map[t, j]] = w[t, j] dout[t],
//                      dw[t, j] = <dout[t], rows[c_map[t, j]]>, 0 at -1
// (the shapes of "[SGLang] CUTLASS MoE", sections 2 and 5, in the rows' own
// type).  Sums are in 32 bits, j ascending.  All are bound by the rows they
// read and write: a token's row is read once, each expert row once.
//
// Rows off the 16-byte grid start at different places between its points, so a
// thread takes a whole piece of what is written (and of what lies like it) and
// puts the other side's columns together from the two pieces they lie across.
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

// Bytes sh .. sh + 15 of the pieces a, b; sh in [0, 16), a multiple of 2.
__device__ __forceinline__ uint4 across(uint4 a, uint4 b, uint32_t sh) {
    const bool by8 = sh & 8, by4 = sh & 4;
    const uint32_t u0 = by8 ? a.z : a.x, u1 = by8 ? a.w : a.y, u2 = by8 ? b.x : a.z, u3 = by8 ? b.y : a.w,
                   u4 = by8 ? b.z : b.x, u5 = by8 ? b.w : b.y;
    const uint32_t v0 = by4 ? u1 : u0, v1 = by4 ? u2 : u1, v2 = by4 ? u3 : u2, v3 = by4 ? u4 : u3, v4 = by4 ? u5 : u4;
    const uint32_t bits = (sh & 3) * 8;
    return make_uint4(__funnelshift_r(v0, v1, bits), __funnelshift_r(v1, v2, bits), __funnelshift_r(v2, v3, bits),
                      __funnelshift_r(v3, v4, bits));
}

// kVe elements from element e on, all of which are in the tensor of `total`
// elements (which starts on the grid).
template <typename T, int LIE>
__device__ __forceinline__ void load_from(Vec<T, kVe<T, LIE>>& v, const T* tensor, int64_t e, int64_t total) {
    if constexpr (LIE == kOff) {
        constexpr int VE = kFull<T>;
        const int64_t piece = e / VE * VE;
        const int se = static_cast<int>(e - piece);
        Vec<T, VE> a, b;
        a.load(tensor + piece);
        b.w = a.w;
        if (se) {
            if (piece + 2 * VE <= total) {
                b.load(tensor + piece + VE);
            } else {  // the tensor ends inside the second piece
                float f[VE];
#pragma unroll
                for (int u = 0; u < VE; ++u) f[u] = piece + VE + u < total ? to_f32(tensor[piece + VE + u]) : 0.f;
                b.set(f);
            }
        }
        v.w = across(a.w, b.w, se * static_cast<uint32_t>(sizeof(T)));
    } else {
        v.load(tensor + e);
    }
}

// CTA (token, chunk of columns): the chunk is read once (off the grid, again
// from L1 for each row) and written to the token's rows.
template <typename T, int LIE>
__global__ void __launch_bounds__(kTokThreads) permute_kernel(TokenParams p) {
    constexpr int VE = kVe<T, LIE>;
    __shared__ int s_row[kMaxSlots];
    const int64_t t = blockIdx.x, total = static_cast<int64_t>(p.T) * p.H;
    load_slots(p, t, s_row);
    const T* src = static_cast<const T*>(p.src);
    const int c0 = (blockIdx.y * kTokThreads + threadIdx.x) * VE;
    Vec<T, VE> v;
    if (LIE != kOff) {
        if (c0 >= p.H) return;
        v.load(src + t * p.H + c0);
    }
    for (int j = 0; j < p.kp; ++j) {
        const int64_t r = s_row[j];
        if (r < 0) continue;
        const int c = c0 - before<T, LIE>(r * p.H);
        T* dst = static_cast<T*>(p.dst) + r * p.H + c;
        if (whole<T, LIE>(c, p.H)) {
            if (LIE == kOff) load_from<T, LIE>(v, src, t * p.H + c, total);
            v.store(dst);
        } else if (LIE == kOff) {
#pragma unroll
            for (int u = 0; u < VE; ++u)
                if (c + u >= 0 && c + u < p.H) dst[u] = src[t * p.H + c + u];
        }
    }
}

constexpr int kRowBatch = 4;  // rows in flight per thread

template <typename T, int LIE>
__global__ void __launch_bounds__(kTokThreads) unpermute_kernel(TokenParams p) {
    constexpr int VE = kVe<T, LIE>;
    __shared__ int s_row[kMaxSlots];
    __shared__ float s_w[kMaxSlots];
    const int64_t t = blockIdx.x, total = static_cast<int64_t>(p.T) * p.kp * p.H;
    if (threadIdx.x < p.kp) s_w[threadIdx.x] = p.w ? p.w[t * p.kp + threadIdx.x] : 1.f;
    load_slots(p, t, s_row);
    const T* src = static_cast<const T*>(p.src);
    const int c = (blockIdx.y * kTokThreads + threadIdx.x) * VE - before<T, LIE>(t * p.H);
    if (c >= p.H) return;
    float acc[VE];
#pragma unroll
    for (int u = 0; u < VE; ++u) acc[u] = 0.f;
    T* dst = static_cast<T*>(p.dst) + t * p.H + c;
    if (whole<T, LIE>(c, p.H)) {
        for (int j0 = 0; j0 < p.kp; j0 += kRowBatch) {
            Vec<T, VE> v[kRowBatch];
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) {
                const int64_t r = j0 + b < p.kp ? s_row[j0 + b] : -1;
                if (r >= 0) load_from<T, LIE>(v[b], src, r * p.H + c, total);
            }
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) {
                if (j0 + b >= p.kp || s_row[j0 + b] < 0) continue;  // a slot without a row adds nothing
                float f[VE];
                v[b].get(f);
#pragma unroll
                for (int u = 0; u < VE; ++u) acc[u] += s_w[j0 + b] * f[u];
            }
        }
        Vec<T, VE> o;
        o.set(acc);
        o.store(dst);
    } else if (LIE == kOff) {
        for (int j = 0; j < p.kp; ++j) {
            const int64_t r = s_row[j];
            if (r < 0) continue;
#pragma unroll
            for (int u = 0; u < VE; ++u)
                if (c + u >= 0 && c + u < p.H) acc[u] += s_w[j] * to_f32(src[r * p.H + c + u]);
        }
#pragma unroll
        for (int u = 0; u < VE; ++u)
            if (c + u >= 0 && c + u < p.H) dst[u] = from_f32<T>(acc[u]);
    }
}

constexpr int kGradTokThreads = 256;

// CTA (token, group of `per` slots): a routing weight's gradient is a sum over
// the whole row, the warps' parts of it gather in shared memory.
template <typename T, int LIE>
__global__ void __launch_bounds__(kGradTokThreads) unpermute_grad_kernel(TokenParams p, int per) {
    constexpr int VE = kVe<T, LIE>, kWarps = kGradTokThreads / 32;
    __shared__ int s_row[kMaxSlots];
    __shared__ float s_w[kMaxSlots];
    __shared__ float s_dot[kMaxSlots][kWarps];
    const int64_t t = blockIdx.x, total = static_cast<int64_t>(p.T) * p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j_begin = blockIdx.y * per, j_end = min(p.kp, j_begin + per);
    const T *src = static_cast<const T*>(p.src), *dout = static_cast<const T*>(p.dout);
    if (threadIdx.x < p.kp) s_w[threadIdx.x] = p.w[t * p.kp + threadIdx.x];
    for (int i = threadIdx.x; i < kMaxSlots * kWarps; i += kGradTokThreads) s_dot[i / kWarps][i % kWarps] = 0.f;
    load_slots(p, t, s_row);
    const int span = p.H + (LIE == kOff ? VE - 1 : 0);
    for (int c0 = threadIdx.x * VE; c0 - static_cast<int>(threadIdx.x) * VE < span; c0 += kGradTokThreads * VE) {
        float d[VE];
        if (LIE != kOff) {
#pragma unroll
            for (int u = 0; u < VE; ++u) d[u] = 0.f;
            if (c0 < p.H) {
                Vec<T, VE> v;
                v.load(dout + t * p.H + c0);
                v.get(d);
            }
        }
        for (int j0 = j_begin; j0 < j_end; j0 += kRowBatch) {
            Vec<T, VE> y[kRowBatch];
            int c[kRowBatch];
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) {
                const int64_t r = j0 + b < j_end ? s_row[j0 + b] : -1;
                c[b] = c0 - (r >= 0 ? before<T, LIE>(r * p.H) : 0);
                if (r >= 0 && whole<T, LIE>(c[b], p.H)) y[b].load(src + r * p.H + c[b]);
            }
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) {
                const int64_t r = j0 + b < j_end ? s_row[j0 + b] : -1;
                if (r < 0) continue;  // the same for the whole CTA
                const float w = s_w[j0 + b];
                float dot = 0.f;
                T* dst = static_cast<T*>(p.dst) + r * p.H + c[b];
                if (whole<T, LIE>(c[b], p.H)) {
                    float f[VE];
                    Vec<T, VE> o;
                    if (LIE == kOff) {
                        load_from<T, LIE>(o, dout, t * p.H + c[b], total);
                        o.get(d);
                    }
                    y[b].get(f);
#pragma unroll
                    for (int u = 0; u < VE; ++u) {
                        dot += d[u] * f[u];
                        f[u] = w * d[u];
                    }
                    o.set(f);
                    o.store(dst);
                } else if (LIE == kOff) {
#pragma unroll
                    for (int u = 0; u < VE; ++u)
                        if (c[b] + u >= 0 && c[b] + u < p.H) {
                            const float g = to_f32(dout[t * p.H + c[b] + u]);
                            dot += g * to_f32(src[r * p.H + c[b] + u]);
                            dst[u] = from_f32<T>(w * g);
                        }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (lane == 0) s_dot[j0 + b][warp] += dot;
            }
        }
    }
    __syncthreads();
    const int j = j_begin + threadIdx.x;
    if (j < j_end) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += s_dot[j][i];
        p.dw[t * p.kp + j] = s;
    }
}

template <typename T, int LIE>
dim3 token_grid(const TokenParams& p) {
    return dim3(p.T, (accesses<T, LIE>(p.H) + kTokThreads - 1) / kTokThreads);
}

}  // namespace

cudaError_t launch_permute(const TokenParams& p, int dtype, int lie, cudaStream_t st) {
    return by_type(dtype, lie, [&](auto t, auto l) {
        using T = decltype(t);
        return launch_kernel(permute_kernel<T, l.value>, token_grid<T, l.value>(p), dim3(kTokThreads), 0, st, false, p);
    });
}

cudaError_t launch_unpermute(const TokenParams& p, int dtype, int lie, cudaStream_t st) {
    return by_type(dtype, lie, [&](auto t, auto l) {
        using T = decltype(t);
        return launch_kernel(unpermute_kernel<T, l.value>, token_grid<T, l.value>(p), dim3(kTokThreads), 0, st, false,
                             p);
    });
}

cudaError_t launch_unpermute_grad(const TokenParams& p, int dtype, int lie, cudaStream_t st) {
    // few tokens: a CTA for each batch of slots
    const int per = p.T < 2 * kSms ? kRowBatch : p.kp;
    return by_type(dtype, lie, [&](auto t, auto l) {
        return launch_kernel(unpermute_grad_kernel<decltype(t), l.value>, dim3(p.T, (p.kp + per - 1) / per),
                             dim3(kGradTokThreads), 0, st, false, p, per);
    });
}

}  // namespace moe
