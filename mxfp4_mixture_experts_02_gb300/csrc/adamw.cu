// AdamW over many tensors in one launch:
//   g' = g c                      (c: an optional scale on the device)
//   m  = m + (1 - b1) (g' - m),   v = v + (1 - b2) (g'^2 - v)
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// m and v are rounded operation by operation, as the formulas are written, so
// the states follow from them alone.
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
constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;

// SplitMix64's output function at state z.
__device__ __forceinline__ uint64_t mix64(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

__device__ __forceinline__ float2 pair(const float (&v)[kE], int k) { return make_float2(v[2 * k], v[2 * k + 1]); }
__device__ __forceinline__ void put_pair(float (&v)[kE], int k, float2 a) {
    v[2 * k] = a.x;
    v[2 * k + 1] = a.y;
}

// a - b, rounded once
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }

// Eight E4M3 codes times 2^(scale code - 127).
__device__ __forceinline__ void decode8(float (&f)[kE], uint2 c, uint32_t scale) {
    const float s = __uint_as_float(scale << 23);
#pragma unroll
    for (int k = 0; k < kE / 2; ++k) {
        const uint32_t two = (k < 2 ? c.x : c.y) >> (16 * (k & 1));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
        put_pair(f, k, mul2(__half22float2(__half2(h)), both(s)));
    }
}

// The exponent of a block's scale from the bits of its largest magnitude, and
// for the roots from those of the largest square: floor(log2 sqrt(v)) is half
// of floor(log2 v), rounded down.
__device__ __forceinline__ int exponent_of(uint32_t amax) { return max(static_cast<int>(amax >> 23) - 134, -126); }
__device__ __forceinline__ int root_exponent_of(uint32_t vmax) {
    if (vmax == 0) return -126;
    const int e = vmax < 0x00800000u ? -118 - __clz(vmax) : static_cast<int>(vmax >> 23) - 127;
    return (e >> 1) - 7;
}

// The codes of eight values, rounded at random.  Divided by 2^120 an E4M3
// number becomes the fp32 number whose exponent and three leading mantissa bits
// are its code, below 2^-6 too, where both stop normalising: so the random
// bits are added to the 20 bits that are cut off.  x = value / scale, at most
// 256 (and a rounding) in magnitude; r: the random bits, `high` half of each.
template <bool SIGNED, bool HIGH>
__device__ __forceinline__ uint2 encode8(const float (&v)[kE], float inv, const uint32_t (&r)[kE]) {
    uint32_t q[kE];
#pragma unroll
    for (int k = 0; k < kE / 2; ++k) {
        const float2 y = mul2(mul2(pair(v, k), both(inv)), both(__uint_as_float(7u << 23)));
        const uint32_t r0 = HIGH ? r[2 * k] >> 16 : r[2 * k] & 0xFFFFu;
        const uint32_t r1 = HIGH ? r[2 * k + 1] >> 16 : r[2 * k + 1] & 0xFFFFu;
        q[2 * k] = __float_as_uint(y.x) + (r0 << 4);
        q[2 * k + 1] = __float_as_uint(y.y) + (r1 << 4);
        if (!SIGNED) {  // what is not zero keeps the smallest code
            q[2 * k] = max(q[2 * k], min(__float_as_uint(v[2 * k]), 1u << 20));
            q[2 * k + 1] = max(q[2 * k + 1], min(__float_as_uint(v[2 * k + 1]), 1u << 20));
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t* a = q + 4 * h;
        // bits 27 .. 20 (27 is zero) to the top byte, four together
        w[h] = __byte_perm(__byte_perm(a[0] << 4, a[1] << 4, 0x0073), __byte_perm(a[2] << 4, a[3] << 4, 0x0073), 0x5410);
        if (SIGNED)
            w[h] |= __byte_perm(__byte_perm(a[0], a[1], 0x0073), __byte_perm(a[2], a[3], 0x0073), 0x5410) & 0x80808080u;
    }
    return make_uint2(w[0], w[1]);
}

// Takes out what is not finite: those of the eight become zero, and NaN codes
// in the answer, to be put over the codes.
__device__ __forceinline__ uint2 take_out_nan(float (&v)[kE]) {
    uint2 nan = make_uint2(0u, 0u);
#pragma unroll
    for (int u = 0; u < kE; ++u)
        if (!(fabsf(v[u]) <= 3.4e38f)) {
            (u < 4 ? nan.x : nan.y) |= 0x7Fu << (8 * (u & 3));
            v[u] = 0.f;
        }
    return nan;
}

// The largest bits of the block's magnitudes, over the four threads that hold
// it.  Bits of magnitudes order as these do, with NaN on top.
__device__ __forceinline__ uint32_t block_max(const float (&v)[kE], uint32_t lanes) {
    uint32_t a = 0u;
#pragma unroll
    for (int u = 0; u < kE; ++u) a = max(a, __float_as_uint(fabsf(v[u])));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) a = max(a, __shfl_xor_sync(lanes, a, o));
    return a;
}

// Eight consecutive elements in accesses of 32 bytes (neighbouring threads then
// fill whole lines) or, from a 16-byte boundary, of 16.
__device__ __forceinline__ void load8(float (&g)[kE], const float* p, bool by32) {
    if (by32) {
        ptx::ld_global_32(g, p);
        return;
    }
#pragma unroll
    for (int i = 0; i < kE; i += 4) {
        Vec<float, 4> v;
        float f[4];
        v.load(p + i);
        v.get(f);
#pragma unroll
        for (int u = 0; u < 4; ++u) g[i + u] = f[u];
    }
}
__device__ __forceinline__ void load8(float (&g)[kE], const __nv_bfloat16* p, bool) {
    Vec<__nv_bfloat16, 8> v;
    v.load(p);
    v.get(g);
}

// Elements i .. i + live - 1 one by one, zeros behind them.
template <typename G>
__device__ __forceinline__ void load_some(float (&g)[kE], const G* p, int live) {
#pragma unroll
    for (int u = 0; u < kE; ++u) g[u] = u < live ? to_f32(p[u]) : 0.f;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[kE], bool by32) {
    if (by32) {
        ptx::st_global_32(p, v);
        return;
    }
#pragma unroll
    for (int u = 0; u < kE; u += 4)
        *reinterpret_cast<float4*>(p + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
}

__device__ __forceinline__ void store_some(float* p, const float (&v)[kE], int live) {
#pragma unroll
    for (int u = 0; u < kE; ++u)
        if (u < live) p[u] = v[u];
}

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int live, bool wide) {
    if (wide) return *reinterpret_cast<const uint2*>(p);
    uint2 c = make_uint2(0u, 0u);
#pragma unroll
    for (int u = 0; u < kE; ++u)
        if (u < live) (u < 4 ? c.x : c.y) |= static_cast<uint32_t>(p[u]) << (8 * (u & 3));
    return c;
}

__device__ __forceinline__ void store_codes(uint8_t* p, uint2 c, int live, bool wide) {
    if (wide) {
        *reinterpret_cast<uint2*>(p) = c;
        return;
    }
#pragma unroll
    for (int u = 0; u < kE; ++u)
        if (u < live) p[u] = static_cast<uint8_t>((u < 4 ? c.x : c.y) >> (8 * (u & 3)));
}

template <typename G, bool MX, int N>
__global__ void __launch_bounds__(kAdamwThreads, 4) adamw_kernel(const __grid_constant__ AdamwBatch<N> b) {
    float clip = 1.f;
    if (b.grad_scale) {
        clip = *b.grad_scale;
        if (!isfinite(clip)) return;  // a gradient that overflowed: the step is skipped
    }
    // the CTA's items lie one behind the other; the first one's tensor is the
    // last that starts at or before it
    const uint32_t per = (b.items + gridDim.x - 1) / gridDim.x;
    const uint32_t first = blockIdx.x * per, last = min(first + per, b.items);
    int at = 0;
    for (int lo = 0, hi = b.count - 1; lo < hi; at = lo) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.t[mid].first_item <= first) lo = mid;
        else hi = mid - 1;
    }
    for (uint32_t item = first; item < last; ++item) {
        while (at + 1 < b.count && b.t[at + 1].first_item <= item) ++at;
        const AdamwTensor& t = b.t[at];
        {
            const int64_t i = static_cast<int64_t>(item - t.first_item) * kAdamwItem + threadIdx.x * kE;
            const int live = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(kE), t.n - i)));
            const bool wide = t.vec && live == kE, by32 = t.vec == 2;
            const G* gp = static_cast<const G*>(t.g) + i;
            float *fm = static_cast<float*>(t.m) + i, *fv = static_cast<float*>(t.v) + i;
            uint8_t *cm = static_cast<uint8_t*>(t.m) + i, *cv = static_cast<uint8_t*>(t.v) + i;
            float p[kE], g[kE], m[kE], v[kE];
            if (wide) {
                load8(p, t.p + i, by32);
                load8(g, gp, by32);
            } else {
                load_some(p, t.p + i, live);
                load_some(g, gp, live);
            }
            if (MX) {
                const uint32_t sm = live ? t.ms[i >> 5] : 0u, sv = live ? t.vs[i >> 5] : 0u;
                decode8(m, load_codes(cm, live, wide), sm);
                decode8(v, load_codes(cv, live, wide), sv);
#pragma unroll
                for (int k = 0; k < kE / 2; ++k) put_pair(v, k, mul2(pair(v, k), pair(v, k)));
            } else if (wide) {
                load8(m, fm, by32);
                load8(v, fv, by32);
            } else {
                load_some(m, fm, live);
                load_some(v, fv, live);
            }
            float root[kE];
#pragma unroll
            for (int k = 0; k < kE / 2; ++k) {
                const float2 g2 = b.grad_scale ? mul2(pair(g, k), both(clip)) : pair(g, k);
                const float2 m2 = add2(pair(m, k), mul2(sub2(g2, pair(m, k)), both(b.one_minus_beta1)));
                const float2 v2 = add2(pair(v, k), mul2(sub2(mul2(g2, g2), pair(v, k)), both(b.one_minus_beta2)));
                // the root and the quotient to within two units in the last
                // place: p moves by lr of it
                const float2 r2 = make_float2(ptx::sqrt_approx(v2.x), ptx::sqrt_approx(v2.y));
                const float2 den = fma2(r2, both(b.inv_root_bc2), both(b.eps));
                const float2 q = make_float2(__fdividef(m2.x, den.x), __fdividef(m2.y, den.y));
                put_pair(m, k, m2);
                put_pair(v, k, v2);
                put_pair(root, k, r2);
                put_pair(p, k, fma2(q, both(-b.step_size), mul2(pair(p, k), both(b.decay))));
            }
            if (wide) store8(t.p + i, p, by32);
            else store_some(t.p + i, p, live);
            if (MX) {
                uint32_t am = block_max(m, 0xffffffffu), av = block_max(v, 0xffffffffu);
                uint2 m_nan = make_uint2(0u, 0u), v_nan = m_nan;
                if (max(am, av) >= 0x7F800000u) {  // the same for the block's threads
                    const uint32_t four = 0xFu << (threadIdx.x & 28);
                    m_nan = take_out_nan(m);
                    v_nan = take_out_nan(v);
                    take_out_nan(root);
                    am = block_max(m, four);
                    av = block_max(v, four);
                }
                // elements 2k and 2k + 1 take the halves of number k + 1
                uint32_t r[kE];
                uint64_t z = b.seed + ((static_cast<uint64_t>(t.counter + i) >> 1) + 1) * kGamma;
#pragma unroll
                for (int u = 0; u < kE; u += 2, z += kGamma) {
                    const uint64_t x = mix64(z);
                    r[u] = static_cast<uint32_t>(x);
                    r[u + 1] = static_cast<uint32_t>(x >> 32);
                }
                const int em = exponent_of(am), ev = root_exponent_of(av);
                uint2 c = encode8<true, false>(m, __uint_as_float(static_cast<uint32_t>(127 - em) << 23), r);
                uint2 d = encode8<false, true>(root, __uint_as_float(static_cast<uint32_t>(127 - ev) << 23), r);
                c.x |= m_nan.x, c.y |= m_nan.y, d.x |= v_nan.x, d.y |= v_nan.y;
                store_codes(cm, c, live, wide);
                store_codes(cv, d, live, wide);
                if (live && (i & 31) == 0) {
                    t.ms[i >> 5] = static_cast<uint8_t>(em + 127);
                    t.vs[i >> 5] = static_cast<uint8_t>(ev + 127);
                }
            } else if (wide) {
                store8(fm, m, by32);
                store8(fv, v, by32);
            } else {
                store_some(fm, m, live);
                store_some(fv, v, live);
            }
        }
    }
}

}  // namespace

template <int N>
cudaError_t launch_adamw(const AdamwBatch<N>& b, int g_dtype, bool mx, cudaStream_t st) {
    const dim3 grid(b.items < kSms * 4u ? b.items : kSms * 4u);
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kAdamwThreads), 0, st, false, b); };
    if (g_dtype == MOE_DTYPE_F32) return mx ? go(adamw_kernel<float, true, N>) : go(adamw_kernel<float, false, N>);
    return mx ? go(adamw_kernel<__nv_bfloat16, true, N>) : go(adamw_kernel<__nv_bfloat16, false, N>);
}

template cudaError_t launch_adamw<kAdamwFew>(const AdamwBatch<kAdamwFew>&, int, bool, cudaStream_t);
template cudaError_t launch_adamw<kAdamwMany>(const AdamwBatch<kAdamwMany>&, int, bool, cudaStream_t);

}  // namespace moe
