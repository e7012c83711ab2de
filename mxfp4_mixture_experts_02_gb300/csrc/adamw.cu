// AdamW over many tensors in one launch:
//   g' = g c                      (c: an optional scale on the device)
//   m  = m + (1 - b1) (g' - m),   v = v + (1 - b2) (g'^2 - v)
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every operation is rounded by itself (no contraction), so the 8-bit codes
// follow from the formulas alone.
//
// 8-bit states: m and sqrt(v) as E4M3 codes with one power-of-two scale per
// 32 values, 2^e with e = floor(log2 max) - 7 (the largest magnitude lies in
// [128, 256), so nothing saturates).  The square root halves the exponent
// range that the second moment needs.  Codes are rounded up or down at random
// in proportion to the distance: the second moment moves by (1 - b2) of its
// distance a step, far less than half a code, and would stand still under
// rounding to nearest.  A root that is not zero keeps at least the smallest
// code, so that no m is divided by eps alone.
#include "train.cuh"

namespace moe {

namespace {

constexpr int kAdamwThreads = 256;
constexpr int kE = 8;  // elements per thread: four threads share a block of 32

// SplitMix64's output function at state z.
__device__ __forceinline__ uint64_t mix64(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// x (|x| < 256) to an E4M3 code with 16 random bits: the 20 mantissa bits
// below E4M3's three are compared with the random bits by an add and cut off.
// Below 2^-6 E4M3's steps stop shrinking at 2^-9; moved up by 2^-6 a value's
// own steps have that size.
__device__ __forceinline__ float e4m3_random(float x, uint32_t r16) {
    float a = fabsf(x);
    if (!(a <= 3.0e38f)) return __uint_as_float(0x7FC00000u);  // no E4M3 infinity: stored as NaN
    const float lift = a < 0.015625f ? 0.015625f : 0.f;
    a = __fadd_rn(a, lift);
    a = __uint_as_float((__float_as_uint(a) + (r16 << 4)) & ~0xFFFFFu);
    return copysignf(__fsub_rn(a, lift), x);
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t c) {
    const float v = e4m3_pos_to_float(c & 127u);
    return (c & 128u) ? -v : v;
}

// The scale exponent of a block with largest magnitude amax.
__device__ __forceinline__ int state_exponent(float amax) {
    const int e = mx_shared_exponent(amax, 7);
    return e < -126 ? -126 : (e > 126 ? 126 : e);
}

template <typename G>
__device__ __forceinline__ void load8(float (&g)[kE], const G* p) {
#pragma unroll
    for (int i = 0; i < kE; i += kFull<G>) {
        Vec<G, kFull<G>> v;
        float f[kFull<G>];
        v.load(p + i);
        v.get(f);
#pragma unroll
        for (int u = 0; u < kFull<G>; ++u) g[i + u] = f[u];
    }
}

template <typename G, bool MX>
__global__ void __launch_bounds__(kAdamwThreads) adamw_kernel(const __grid_constant__ AdamwBatch<kAdamwMaxTensors> b) {
    __shared__ int s_tensor;
    float clip = 1.f;
    if (b.grad_scale) {
        clip = *b.grad_scale;
        if (!isfinite(clip)) return;  // a gradient that overflowed: the step is skipped
    }
    for (uint32_t item = blockIdx.x; item < b.items; item += gridDim.x) {
        if (threadIdx.x == 0) {  // the last tensor that starts at or before the item
            int lo = 0, hi = b.count - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (b.t[mid].first_item <= item) lo = mid;
                else hi = mid - 1;
            }
            s_tensor = lo;
        }
        __syncthreads();
        const AdamwTensor& t = b.t[s_tensor];
        const int64_t begin = static_cast<int64_t>(item - t.first_item) * kAdamwItem;
        const int64_t end = min(begin + kAdamwItem, t.n);
        const G* gp = static_cast<const G*>(t.g);
        for (int64_t i0 = begin; i0 < end; i0 += kAdamwThreads * kE) {
            const int64_t i = i0 + threadIdx.x * kE;
            const int live = i < end ? static_cast<int>(min(static_cast<int64_t>(kE), end - i)) : 0;
            const bool wide = t.vec && live == kE;
            float p[kE], g[kE], m[kE], v[kE];
            if (wide) {
                load8(p, t.p + i);
                load8(g, gp + i);
            } else {
#pragma unroll
                for (int u = 0; u < kE; ++u) {
                    p[u] = u < live ? t.p[i + u] : 0.f;
                    g[u] = u < live ? to_f32(gp[i + u]) : 0.f;
                }
            }
            if (MX) {
                const uint8_t* mc = static_cast<const uint8_t*>(t.m);
                const uint8_t* vc = static_cast<const uint8_t*>(t.v);
                float sm = 0.f, sv = 0.f;
                if (live) {
                    sm = exp2_int(t.ms[i >> 5] - 127);
                    sv = exp2_int(t.vs[i >> 5] - 127);
                }
                if (wide) {
                    const uint2 cm = *reinterpret_cast<const uint2*>(mc + i), cv = *reinterpret_cast<const uint2*>(vc + i);
#pragma unroll
                    for (int u = 0; u < kE; ++u) {
                        m[u] = __fmul_rn(e4m3_to_f32(((u < 4 ? cm.x : cm.y) >> (8 * (u & 3))) & 255u), sm);
                        v[u] = __fmul_rn(e4m3_to_f32(((u < 4 ? cv.x : cv.y) >> (8 * (u & 3))) & 255u), sv);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < kE; ++u) {
                        m[u] = u < live ? __fmul_rn(e4m3_to_f32(mc[i + u]), sm) : 0.f;
                        v[u] = u < live ? __fmul_rn(e4m3_to_f32(vc[i + u]), sv) : 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < kE; ++u) v[u] = __fmul_rn(v[u], v[u]);
            } else if (wide) {
                load8(m, static_cast<const float*>(t.m) + i);
                load8(v, static_cast<const float*>(t.v) + i);
            } else {
#pragma unroll
                for (int u = 0; u < kE; ++u) {
                    m[u] = u < live ? static_cast<const float*>(t.m)[i + u] : 0.f;
                    v[u] = u < live ? static_cast<const float*>(t.v)[i + u] : 0.f;
                }
            }
            float root[kE];
#pragma unroll
            for (int u = 0; u < kE; ++u) {
                const float gc = b.grad_scale ? __fmul_rn(g[u], clip) : g[u];
                m[u] = __fadd_rn(m[u], __fmul_rn(__fsub_rn(gc, m[u]), b.one_minus_beta1));
                v[u] = __fadd_rn(v[u], __fmul_rn(__fsub_rn(__fmul_rn(gc, gc), v[u]), b.one_minus_beta2));
                root[u] = __fsqrt_rn(v[u]);
                const float den = __fadd_rn(__fmul_rn(root[u], b.inv_root_bc2), b.eps);
                p[u] = __fsub_rn(__fmul_rn(p[u], b.decay), __fmul_rn(__fdiv_rn(m[u], den), b.step_size));
            }
            if (wide) {
#pragma unroll
                for (int u = 0; u < kE; u += 4)
                    *reinterpret_cast<float4*>(t.p + i + u) = make_float4(p[u], p[u + 1], p[u + 2], p[u + 3]);
            } else {
#pragma unroll
                for (int u = 0; u < kE; ++u)
                    if (u < live) t.p[i + u] = p[u];
            }
            if (MX) {
                float am = 0.f, av = 0.f;
#pragma unroll
                for (int u = 0; u < kE; ++u)
                    if (u < live) am = fmaxf(am, fabsf(m[u])), av = fmaxf(av, root[u]);
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                    av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
                }
                const int em = state_exponent(am), ev = state_exponent(av);
                const float im = exp2_int(-em), iv = exp2_int(-ev);
                uint32_t cm[kE], cv[kE];
#pragma unroll
                for (int u = 0; u < kE; u += 2) {
                    // elements 2k and 2k + 1 take the halves of number k + 1
                    const uint64_t k1 = (static_cast<uint64_t>(t.counter + i + u) >> 1) + 1;
                    const uint64_t r = mix64(b.seed + k1 * 0x9E3779B97F4A7C15ull);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t bits = static_cast<uint32_t>(r >> (32 * w));
                        const float qm = e4m3_random(__fmul_rn(m[u + w], im), bits & 0xFFFFu);
                        float qv = e4m3_random(__fmul_rn(root[u + w], iv), bits >> 16);
                        if (root[u + w] != 0.f && qv < 0.001953125f) qv = 0.001953125f;  // a NaN stays one
                        const uint32_t c = e4m3x2(qm, qv);
                        cm[u + w] = c & 255u;
                        cv[u + w] = c >> 8;
                    }
                }
                uint8_t* mo = static_cast<uint8_t*>(t.m);
                uint8_t* vo = static_cast<uint8_t*>(t.v);
                if (wide) {
                    *reinterpret_cast<uint2*>(mo + i) = make_uint2(cm[0] | cm[1] << 8 | cm[2] << 16 | cm[3] << 24,
                                                                   cm[4] | cm[5] << 8 | cm[6] << 16 | cm[7] << 24);
                    *reinterpret_cast<uint2*>(vo + i) = make_uint2(cv[0] | cv[1] << 8 | cv[2] << 16 | cv[3] << 24,
                                                                   cv[4] | cv[5] << 8 | cv[6] << 16 | cv[7] << 24);
                } else {
#pragma unroll
                    for (int u = 0; u < kE; ++u)
                        if (u < live) mo[i + u] = static_cast<uint8_t>(cm[u]), vo[i + u] = static_cast<uint8_t>(cv[u]);
                }
                if (live && (i & 31) == 0) {
                    t.ms[i >> 5] = static_cast<uint8_t>(em + 127);
                    t.vs[i >> 5] = static_cast<uint8_t>(ev + 127);
                }
            } else if (wide) {
                float *mo = static_cast<float*>(t.m) + i, *vo = static_cast<float*>(t.v) + i;
#pragma unroll
                for (int u = 0; u < kE; u += 4) {
                    *reinterpret_cast<float4*>(mo + u) = make_float4(m[u], m[u + 1], m[u + 2], m[u + 3]);
                    *reinterpret_cast<float4*>(vo + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kE; ++u)
                    if (u < live) static_cast<float*>(t.m)[i + u] = m[u], static_cast<float*>(t.v)[i + u] = v[u];
            }
        }
        __syncthreads();  // s_tensor is read until here
    }
}

}  // namespace

cudaError_t launch_adamw(const AdamwBatch<kAdamwMaxTensors>& b, int g_dtype, bool mx, cudaStream_t st) {
    const dim3 grid(b.items < kSms * 8u ? b.items : kSms * 8u);
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kAdamwThreads), 0, st, false, b); };
    if (g_dtype == MOE_DTYPE_F32) return mx ? go(adamw_kernel<float, true>) : go(adamw_kernel<float, false>);
    return mx ? go(adamw_kernel<__nv_bfloat16, true>) : go(adamw_kernel<__nv_bfloat16, false>);
}

}  // namespace moe
