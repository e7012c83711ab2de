// Parameter blocks, launchers and typed loads of the training operators
// around the experts: layer norm, permute / unpermute, the routing gradient
// and AdamW.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {

// ------------------------------------------------------------ typed vectors
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}

// Elements of a 16-byte access.
template <typename T>
constexpr int kFull = 16 / static_cast<int>(sizeof(T));

// N elements moved with one access of their whole size: one element, or 16
// bytes kept as packed words (16-bit elements apart cost a register each).
// Never wider: sm_103a has 32-byte accesses, which fault on the 16-byte
// boundary that the entries check.
template <typename T, int N>
struct Vec {
    static_assert(N == kFull<T>, "one element or 16 bytes");
    uint4 w;
    __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = w; }
    __device__ __forceinline__ void get(float (&f)[N]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(u[i]);
            } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                f[2 * i] = h.x;
                f[2 * i + 1] = h.y;
            }
        }
    }
    // rounded to nearest even
    __device__ __forceinline__ void set(const float (&f)[N]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                u[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        w = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = from_f32<T>(f[0]); }
};

// Two fp32 operations in one instruction, each half rounded by itself.
__device__ __forceinline__ uint64_t bits2(float2 a) {
    return static_cast<uint64_t>(__float_as_uint(a.x)) | static_cast<uint64_t>(__float_as_uint(a.y)) << 32;
}
__device__ __forceinline__ float2 float2_of(uint64_t b) {
    return make_float2(__uint_as_float(static_cast<uint32_t>(b)), __uint_as_float(static_cast<uint32_t>(b >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return float2_of(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// How rows lie in memory:
//   kGrid    every row starts on the 16-byte grid
//   kOff     the tensors start on the grid, their rows do not (a row length
//            that is no multiple of 16 bytes); a thread takes a whole piece of
//            the grid, and the pieces at the ends of a row reach over them
//   kSingle  element by element, for tensors that start off the grid
enum Lie { kGrid, kOff, kSingle };

template <typename T, int LIE>
constexpr int kVe = LIE == kSingle ? 1 : kFull<T>;

// Accesses that a row takes, wherever it starts.
template <typename T, int LIE>
int accesses(int cols) {
    constexpr int VE = kVe<T, LIE>;
    return (cols + VE - 1 + (LIE == kOff ? VE - 1 : 0)) / VE;
}

// Elements of the row from element `first` on that lie before it in its first
// piece of the grid.
template <typename T, int LIE>
__device__ __forceinline__ int before(int64_t first) {
    return LIE == kOff ? static_cast<int>(first % kFull<T>) : 0;
}

// The columns c .. c + VE - 1 are all in the row.
template <typename T, int LIE>
__device__ __forceinline__ bool whole(int c, int cols) {
    return LIE == kOff ? c >= 0 && c + kFull<T> <= cols : c < cols;
}

template <typename F>
cudaError_t by_type(int dtype, int lie, F f) {
    auto go = [&](auto t) {
        if (lie == kGrid) return f(t, std::integral_constant<int, kGrid>{});
        if (lie == kOff) return f(t, std::integral_constant<int, kOff>{});
        return f(t, std::integral_constant<int, kSingle>{});
    };
    return dtype == MOE_DTYPE_BF16 ? go(__nv_bfloat16{}) : dtype == MOE_DTYPE_F16 ? go(__half{}) : go(float{});
}

// N parameters (a norm's weight or bias) from column c on, kept in 32 bits or
// in the rows' type.
template <typename T, int N>
__device__ __forceinline__ void load_param(float (&out)[N], const void* p, bool f32, int64_t c) {
    if (f32) {
        constexpr int M = N < 4 ? N : 4;
#pragma unroll
        for (int i = 0; i < N; i += M) {
            Vec<float, M> v;
            float f[M];
            v.load(static_cast<const float*>(p) + c + i);
            v.get(f);
#pragma unroll
            for (int u = 0; u < M; ++u) out[i + u] = f[u];
        }
    } else {
        Vec<T, N> v;
        v.load(static_cast<const T*>(p) + c);
        v.get(out);
    }
}

// ------------------------------------------------------------ layer norm
struct NormParams {
    const void *x, *residual, *weight, *bias;  // residual, weight, bias may be null
    void *h, *y;                               // h: x + residual (null without a residual)
    float *mean, *rstd;
    int64_t rows;
    int cols, w_f32;
    float eps;
};

struct NormGradParams {
    const void *dy, *h, *weight, *dh;  // weight, dh may be null
    const float *mean, *rstd;
    void* dx;
    float *dweight, *dbias;  // either may be null
    float* partial;          // [grid][2][cols]
    int64_t rows;
    int cols, w_f32;
};

constexpr int kSms = 152;  // streaming multiprocessors of a GB300

// CTAs of the backward pass that own partial column sums.
constexpr int kNormMaxPartials = 4 * kSms;

cudaError_t launch_norm(const NormParams& p, int dtype, int lie, cudaStream_t st);
cudaError_t launch_norm_grad(const NormGradParams& p, int dtype, int lie, cudaStream_t st);

// ------------------------------------------------------------ tokens <-> rows
struct TokenParams {
    const void* src;       // permute: x [T, H]; unpermute: rows
    const void* dout;      // unpermute's gradient: dout [T, H]
    const float* w;        // [T, k'] or null (weight 1)
    const int32_t* c_map;  // [T, k']
    void* dst;
    float* dw;  // [T, k']
    int T, kp, H;
};

// Slots sorted by expert (of p: ids, offsets, a_map, c_map and, for long
// batches, the sort's other tables).
cudaError_t launch_token_map(const SortParams& p, cudaStream_t st);
cudaError_t launch_permute(const TokenParams& p, int dtype, int lie, cudaStream_t st);
cudaError_t launch_unpermute(const TokenParams& p, int dtype, int lie, cudaStream_t st);
cudaError_t launch_unpermute_grad(const TokenParams& p, int dtype, int lie, cudaStream_t st);

// ------------------------------------------------------------ routing gradient
struct RouteGradParams {
    const int32_t* ids;
    const float *w, *dw;
    const uint16_t* shared_logit;
    float *dlogits, *dshared;
    int T, Eg, k, S, kp;
    float shared_scale;
};

cudaError_t launch_route_grad(const RouteGradParams& p, cudaStream_t st);

// ------------------------------------------------------------ AdamW
// One tensor as the kernel sees it: its first work item and the number of its
// first element in the call's random sequence.
struct AdamwTensor {
    float* p;
    const void* g;
    void *m, *v;
    uint8_t *ms, *vs;
    int64_t n;
    int64_t counter;
    uint32_t first_item;
    uint32_t vec;  // 1: every pointer is aligned for 16-byte accesses, 2: and for 32-byte ones; else 0
};

// A launch's tensors travel in its parameters (at most 32764 bytes): the usual
// few, or as many as fit.
constexpr int kAdamwFew = 32, kAdamwMany = 448;

template <int N>
struct AdamwBatch {
    AdamwTensor t[N];
    const float* grad_scale;
    uint64_t seed;
    float one_minus_beta1, one_minus_beta2, decay, step_size, inv_root_bc2, eps;
    uint32_t items;
    int item_elems;  // of a work item: a multiple of kAdamwStep
    int count;
};

static_assert(sizeof(AdamwBatch<kAdamwMany>) <= 32764, "kernel parameters");

constexpr int kAdamwStep = 2048;  // elements that a CTA takes at once: eight for each thread
constexpr int kAdamwItem = 8;     // most steps of a work item

template <int N>
cudaError_t launch_adamw(const AdamwBatch<N>& b, int g_dtype, bool mx, cudaStream_t st);

}  // namespace moe
