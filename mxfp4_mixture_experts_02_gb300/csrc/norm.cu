// Layer norm of the rows in front of the router and the experts, with the
// residual stream's sum in front of it:
//   h = x + r (rounded to the rows' type: the stream is stored so)
//   mean = sum h / n,  rstd = (sum (h - mean)^2 / n + eps)^-1/2
//   y = (h - mean) rstd w + b
// A row is read once and stays in registers, so the variance is the sum of
// squared distances from the mean (no cancellation); sums are in 32 bits.
#include "train.cuh"

namespace moe {

namespace {

// Sum over the L lanes of a sub-warp group (L a power of two, all lanes of
// the warp take part).
__device__ __forceinline__ float lanes_sum(float v, int L) {
    for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the CTA (a multiple of 32 threads) in a fixed order.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
    v = lanes_sum(v, 32);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    return lanes_sum(lane < nw ? s_part[lane] : 0.f, 32);
}

constexpr int kWarpRowThreads = 128;

// V accesses of VE elements per thread hold a row.  WARP: L <= 32 lanes take
// a row, 128 / L rows per CTA; else the CTA takes one row and L = blockDim.x.
template <typename T, int VE, int V, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpRowThreads : 1024) norm_kernel(NormParams p, int L) {
    __shared__ float s_part[2][32];
    const int64_t row = WARP ? (static_cast<int64_t>(blockIdx.x) * kWarpRowThreads + threadIdx.x) / L : blockIdx.x;
    const int lane = WARP ? threadIdx.x & (L - 1) : threadIdx.x;
    const int nvec = p.cols / VE;
    const bool live = row < p.rows;  // lanes past the last row take part in the shuffles
    const int64_t base = row * p.cols;
    const T* x = static_cast<const T*>(p.x) + base;
    Vec<T, VE> h[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (live && i * L + lane < nvec) h[i] = load_vec<T, VE>(x + static_cast<int64_t>(i * L + lane) * VE);
    if (p.residual) {
        const T* r = static_cast<const T*>(p.residual) + base;
        T* ho = static_cast<T*>(p.h) + base;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (live && i * L + lane < nvec) {
                const int64_t c = static_cast<int64_t>(i * L + lane) * VE;
                const Vec<T, VE> a = load_vec<T, VE>(r + c);
#pragma unroll
                for (int u = 0; u < VE; ++u) h[i].v[u] = from_f32<T>(to_f32(h[i].v[u]) + to_f32(a.v[u]));
                store_vec<T, VE>(ho + c, h[i]);
            }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (live && i * L + lane < nvec) {
#pragma unroll
            for (int u = 0; u < VE; ++u) s += to_f32(h[i].v[u]);
        }
    const float inv_n = 1.0f / static_cast<float>(p.cols);
    const float mean = (WARP ? lanes_sum(s, L) : block_sum(s, s_part[0])) * inv_n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (live && i * L + lane < nvec) {
#pragma unroll
            for (int u = 0; u < VE; ++u) {
                const float d = to_f32(h[i].v[u]) - mean;
                q += d * d;
            }
        }
    const float var = (WARP ? lanes_sum(q, L) : block_sum(q, s_part[1])) * inv_n;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (!live) return;
    if (lane == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + base;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i * L + lane < nvec) {
            const int64_t c = static_cast<int64_t>(i * L + lane) * VE;
            float w[VE], b[VE];
#pragma unroll
            for (int u = 0; u < VE; ++u) w[u] = 1.f, b[u] = 0.f;
            if (p.weight) load_param<T, VE>(w, p.weight, p.w_f32, c);
            if (p.bias) load_param<T, VE>(b, p.bias, p.w_f32, c);
            Vec<T, VE> o;
#pragma unroll
            for (int u = 0; u < VE; ++u) o.v[u] = from_f32<T>((to_f32(h[i].v[u]) - mean) * rstd * w[u] + b[u]);
            store_vec<T, VE>(y + c, o);
        }
}

// Rows too long for a CTA's registers: the same three passes, re-reading the
// row (h, where there is a residual) from the caches.
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(NormParams p) {
    __shared__ float s_part[2][32];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * p.cols;
    const T* x = static_cast<const T*>(p.x) + base;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + base : nullptr;
    T* ho = static_cast<T*>(p.h) + base;
    float s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        T v = x[c];
        if (r) ho[c] = v = from_f32<T>(to_f32(v) + to_f32(r[c]));
        s += to_f32(v);
    }
    const T* h = r ? ho : x;  // each thread reads back what it wrote itself
    const float inv_n = 1.0f / static_cast<float>(p.cols);
    const float mean = block_sum(s, s_part[0]) * inv_n;
    float q = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        const float d = to_f32(h[c]) - mean;
        q += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, s_part[1]) * inv_n + p.eps);
    if (threadIdx.x == 0) {
        p.mean[blockIdx.x] = mean;
        p.rstd[blockIdx.x] = rstd;
    }
    T* y = static_cast<T*>(p.y) + base;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float w[1] = {1.f}, b[1] = {0.f};
        if (p.weight) load_param<T, 1>(w, p.weight, p.w_f32, c);
        if (p.bias) load_param<T, 1>(b, p.bias, p.w_f32, c);
        y[c] = from_f32<T>((to_f32(h[c]) - mean) * rstd * w[0] + b[0]);
    }
}

int pow2_at_least(int v) {
    int r = 1;
    while (r < v) r <<= 1;
    return r;
}

template <typename T, int VE, bool WARP>
cudaError_t launch_norm_v(const NormParams& p, int L, int V, cudaStream_t st) {
    const int threads = WARP ? kWarpRowThreads : L;
    const int rows_per_cta = WARP ? kWarpRowThreads / L : 1;
    const dim3 grid(static_cast<unsigned>((p.rows + rows_per_cta - 1) / rows_per_cta));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(threads), 0, st, false, p, L); };
    if (V <= 1) return go(norm_kernel<T, VE, 1, WARP>);
    if (V <= 2) return go(norm_kernel<T, VE, 2, WARP>);
    if (V <= 4) return go(norm_kernel<T, VE, 4, WARP>);
    if (V <= 8) return go(norm_kernel<T, VE, 8, WARP>);
    return go(norm_kernel<T, VE, 16, WARP>);
}

template <typename T, int VE>
cudaError_t launch_norm_t(const NormParams& p, cudaStream_t st) {
    const int nvec = p.cols / VE;
    if (nvec <= 32 * 16) {
        const int L = nvec >= 32 ? 32 : pow2_at_least(nvec);
        return launch_norm_v<T, VE, true>(p, L, (nvec + L - 1) / L, st);
    }
    if (nvec <= 1024 * 4) {
        const int L = ((nvec + 3) / 4 + 31) & ~31;
        return launch_norm_v<T, VE, false>(p, L, 4, st);
    }
    return launch_kernel(norm_long_kernel<T>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, false, p);
}

// ------------------------------------------------------------ gradient
// With xh = (h - mean) rstd and a = dy w:
//   dx = rstd (a - mean(a) - xh mean(a xh)) (+ dh, the residual stream's)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// A CTA walks over rows; a thread owns the same columns of each, so its sums
// of dy xh and dy stay in registers and leave once, as one row of partial
// sums per CTA; a second launch adds those in a fixed order.
constexpr int kGradThreads = 256;  // warp rows

template <typename T, int VE, int V, bool WARP>
__global__ void __launch_bounds__(WARP ? kGradThreads : 1024, 1) norm_grad_kernel(NormGradParams p, int L) {
    __shared__ float s_part[2][2][32];
    extern __shared__ float s_sum[];  // WARP: [2][cols]
    const int lane = WARP ? threadIdx.x & (L - 1) : threadIdx.x;
    const int rows_per_cta = WARP ? kGradThreads / L : 1;
    const int nvec = p.cols / VE;
    const float inv_n = 1.0f / static_cast<float>(p.cols);
    float aw[V * VE], ab[V * VE];
#pragma unroll
    for (int i = 0; i < V * VE; ++i) aw[i] = ab[i] = 0.f;
    int turn = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows_per_cta; r0 < p.rows;
         r0 += static_cast<int64_t>(gridDim.x) * rows_per_cta) {
        const int64_t row = WARP ? r0 + threadIdx.x / L : r0;
        const bool live = row < p.rows;
        const int64_t base = row * p.cols;
        const float mean = live ? p.mean[row] : 0.f, rstd = live ? p.rstd[row] : 0.f;
        Vec<T, VE> x[V], dy[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (live && i * L + lane < nvec) {
                const int64_t c = base + static_cast<int64_t>(i * L + lane) * VE;
                x[i] = load_vec<T, VE>(static_cast<const T*>(p.h) + c);
                dy[i] = load_vec<T, VE>(static_cast<const T*>(p.dy) + c);
            }
        float sa = 0.f, sx = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (live && i * L + lane < nvec) {
                float w[VE];
#pragma unroll
                for (int u = 0; u < VE; ++u) w[u] = 1.f;
                if (p.weight) load_param<T, VE>(w, p.weight, p.w_f32, static_cast<int64_t>(i * L + lane) * VE);
#pragma unroll
                for (int u = 0; u < VE; ++u) {
                    const float g = to_f32(dy[i].v[u]), xh = (to_f32(x[i].v[u]) - mean) * rstd, a = g * w[u];
                    sa += a;
                    sx += a * xh;
                    aw[i * VE + u] += g * xh;
                    ab[i * VE + u] += g;
                }
            }
        if (WARP) {
            sa = lanes_sum(sa, L);
            sx = lanes_sum(sx, L);
        } else {
            // two sets of sums in turn: a set is written again only after the
            // barrier of the row between
            sa = lanes_sum(sa, 32);
            sx = lanes_sum(sx, 32);
            if ((threadIdx.x & 31) == 0) {
                s_part[turn][0][threadIdx.x >> 5] = sa;
                s_part[turn][1][threadIdx.x >> 5] = sx;
            }
            __syncthreads();
            const int nw = blockDim.x >> 5, wl = threadIdx.x & 31;
            sa = lanes_sum(wl < nw ? s_part[turn][0][wl] : 0.f, 32);
            sx = lanes_sum(wl < nw ? s_part[turn][1][wl] : 0.f, 32);
            turn ^= 1;
        }
        const float ma = sa * inv_n, mx = sx * inv_n;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (live && i * L + lane < nvec) {
                const int64_t wc = static_cast<int64_t>(i * L + lane) * VE;
                float w[VE];
#pragma unroll
                for (int u = 0; u < VE; ++u) w[u] = 1.f;
                if (p.weight) load_param<T, VE>(w, p.weight, p.w_f32, wc);
                float o[VE];
#pragma unroll
                for (int u = 0; u < VE; ++u) {
                    const float xh = (to_f32(x[i].v[u]) - mean) * rstd;
                    o[u] = rstd * (to_f32(dy[i].v[u]) * w[u] - ma - xh * mx);
                }
                if (p.dh) {
                    const Vec<T, VE> d = load_vec<T, VE>(static_cast<const T*>(p.dh) + base + wc);
#pragma unroll
                    for (int u = 0; u < VE; ++u) o[u] += to_f32(d.v[u]);
                }
                Vec<T, VE> out;
#pragma unroll
                for (int u = 0; u < VE; ++u) out.v[u] = from_f32<T>(o[u]);
                store_vec<T, VE>(static_cast<T*>(p.dx) + base + wc, out);
            }
    }
    if (!p.partial) return;
    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
    if (!WARP) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * L + lane < nvec) {
                const int c = (i * L + lane) * VE;
#pragma unroll
                for (int u = 0; u < VE; ++u) {
                    part[c + u] = aw[i * VE + u];
                    part[p.cols + c + u] = ab[i * VE + u];
                }
            }
        return;
    }
    // the warp's groups, then the CTA's warps one after another
#pragma unroll
    for (int i = 0; i < V * VE; ++i)
        for (int o = 16; o >= L; o >>= 1) {
            aw[i] += __shfl_xor_sync(0xffffffffu, aw[i], o);
            ab[i] += __shfl_xor_sync(0xffffffffu, ab[i], o);
        }
    const bool first = (threadIdx.x & 31) < L;
    for (int wi = 0; wi < kGradThreads / 32; ++wi) {
        if (first && static_cast<int>(threadIdx.x >> 5) == wi) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * L + lane < nvec) {
                    const int c = (i * L + lane) * VE;
#pragma unroll
                    for (int u = 0; u < VE; ++u) {
                        s_sum[c + u] = (wi ? s_sum[c + u] : 0.f) + aw[i * VE + u];
                        s_sum[p.cols + c + u] = (wi ? s_sum[p.cols + c + u] : 0.f) + ab[i * VE + u];
                    }
                }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * p.cols; c += kGradThreads) part[c] = s_sum[c];
}

// Long rows: dx alone, the row re-read from the caches.
template <typename T>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(NormGradParams p) {
    __shared__ float s_part[2][32];
    const int64_t row = blockIdx.x, base = row * p.cols;
    const T* x = static_cast<const T*>(p.h) + base;
    const T* dy = static_cast<const T*>(p.dy) + base;
    const float mean = p.mean[row], rstd = p.rstd[row], inv_n = 1.0f / static_cast<float>(p.cols);
    float sa = 0.f, sx = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float w[1] = {1.f};
        if (p.weight) load_param<T, 1>(w, p.weight, p.w_f32, c);
        const float a = to_f32(dy[c]) * w[0];
        sa += a;
        sx += a * (to_f32(x[c]) - mean) * rstd;
    }
    const float ma = block_sum(sa, s_part[0]) * inv_n, mx = block_sum(sx, s_part[1]) * inv_n;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float w[1] = {1.f};
        if (p.weight) load_param<T, 1>(w, p.weight, p.w_f32, c);
        const float xh = (to_f32(x[c]) - mean) * rstd;
        float o = rstd * (to_f32(dy[c]) * w[0] - ma - xh * mx);
        if (p.dh) o += to_f32(static_cast<const T*>(p.dh)[base + c]);
        static_cast<T*>(p.dx)[base + c] = from_f32<T>(o);
    }
}

// Long rows: column sums of rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) norm_grad_cols_kernel(NormGradParams p) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float g = to_f32(static_cast<const T*>(p.dy)[row * p.cols + c]);
        const float xh = (to_f32(static_cast<const T*>(p.h)[row * p.cols + c]) - p.mean[row]) * p.rstd[row];
        aw += g * xh;
        ab += g;
    }
    float* part = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.cols;
    part[c] = aw;
    part[p.cols + c] = ab;
}

// Column sums over the partial rows: 32 columns per CTA, 32 threads deep.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(NormGradParams p, int parts) {
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), depth = threadIdx.x >> 5;
    float a = 0.f;
    if (c < 2 * p.cols)
        for (int g = depth; g < parts; g += 32) a += p.partial[static_cast<int64_t>(g) * 2 * p.cols + c];
    s[depth][threadIdx.x & 31] = a;
    __syncthreads();
    const float t = lanes_sum(s[threadIdx.x & 31][depth], 32);  // column `depth` of this CTA's 32
    const int cc = blockIdx.x * 32 + depth;
    if ((threadIdx.x & 31) == 0 && cc < 2 * p.cols) {
        if (cc < p.cols) {
            if (p.dweight) p.dweight[cc] = t;
        } else if (p.dbias) {
            p.dbias[cc - p.cols] = t;
        }
    }
}

template <typename T, int VE, bool WARP>
cudaError_t launch_norm_grad_v(const NormGradParams& p, int L, int V, int grid, cudaStream_t st) {
    const int threads = WARP ? kGradThreads : L;
    const size_t smem = WARP ? size_t(2) * p.cols * sizeof(float) : 0;
    auto go = [&](auto kernel) { return launch_kernel(kernel, dim3(grid), dim3(threads), smem, st, false, p, L); };
    if (V <= 1) return go(norm_grad_kernel<T, VE, 1, WARP>);
    if (V <= 2) return go(norm_grad_kernel<T, VE, 2, WARP>);
    if constexpr (VE * 4 <= 32)
        if (V <= 4) return go(norm_grad_kernel<T, VE, 4, WARP>);
    if constexpr (VE * 8 <= 32)
        if (V <= 8) return go(norm_grad_kernel<T, VE, 8, WARP>);
    if constexpr (VE * 16 <= 32)
        if (V <= 16) return go(norm_grad_kernel<T, VE, 16, WARP>);
    if constexpr (VE * 32 <= 32)
        if (V <= 32) return go(norm_grad_kernel<T, VE, 32, WARP>);
    return cudaErrorInvalidValue;
}

template <typename T, int VE>
cudaError_t launch_norm_grad_t(const NormGradParams& p, cudaStream_t st) {
    const int nvec = p.cols / VE;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (p.rows == 0) {
        // no row: the sums are zero
    } else if (p.cols <= 1024) {  // V * VE <= 32 with 32 lanes
        const int L = nvec >= 32 ? 32 : pow2_at_least(nvec);
        const int64_t ctas = (p.rows + kGradThreads / L - 1) / (kGradThreads / L);
        parts = static_cast<int>(ctas < kNormMaxPartials ? ctas : kNormMaxPartials);
        e = launch_norm_grad_v<T, VE, true>(p, L, (nvec + L - 1) / L, parts, st);
    } else if (p.cols <= 8192) {  // V * VE <= 16 with up to 512 threads
        constexpr int V = 16 / VE;
        const int L = ((nvec + V - 1) / V + 31) & ~31;
        parts = static_cast<int>(p.rows < kNormMaxPartials ? p.rows : kNormMaxPartials);
        e = launch_norm_grad_v<T, VE, false>(p, L, V, parts, st);
    } else {
        // the column sums first: dx may take dy's place
        parts = static_cast<int>(p.rows < 64 ? p.rows : 64);
        if (p.partial)
            e = launch_kernel(norm_grad_cols_kernel<T>, dim3((p.cols + 255) / 256, parts), dim3(256), 0, st, false, p);
        if (e == cudaSuccess)
            e = launch_kernel(norm_grad_long_kernel<T>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, false,
                              p);
    }
    if (e != cudaSuccess || !p.partial) return e;
    return launch_kernel(norm_grad_sum_kernel, dim3((2 * p.cols + 31) / 32), dim3(1024), 0, st, false, p, parts);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int dtype, bool vec, cudaStream_t st) {
    switch (dtype) {
        case MOE_DTYPE_BF16:
            return vec ? launch_norm_t<__nv_bfloat16, 8>(p, st) : launch_norm_t<__nv_bfloat16, 1>(p, st);
        case MOE_DTYPE_F16:
            return vec ? launch_norm_t<__half, 8>(p, st) : launch_norm_t<__half, 1>(p, st);
        default:
            return vec ? launch_norm_t<float, 4>(p, st) : launch_norm_t<float, 1>(p, st);
    }
}

cudaError_t launch_norm_grad(const NormGradParams& p, int dtype, bool vec, cudaStream_t st) {
    switch (dtype) {
        case MOE_DTYPE_BF16:
            return vec ? launch_norm_grad_t<__nv_bfloat16, 8>(p, st) : launch_norm_grad_t<__nv_bfloat16, 1>(p, st);
        case MOE_DTYPE_F16:
            return vec ? launch_norm_grad_t<__half, 8>(p, st) : launch_norm_grad_t<__half, 1>(p, st);
        default:
            return vec ? launch_norm_grad_t<float, 4>(p, st) : launch_norm_grad_t<float, 1>(p, st);
    }
}

}  // namespace moe
