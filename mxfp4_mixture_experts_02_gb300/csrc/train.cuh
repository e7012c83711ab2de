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

// N elements moved with one access of their whole size, at most 16 bytes: the
// alignment that the entries check (sm_103a has 32-byte accesses, which the
// compiler takes for a larger type and which fault on a 16-byte boundary).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    static_assert(sizeof(T) * N <= 16, "wider than the alignment that is checked");
    T v[N];
};

// Elements of a 16-byte access.
template <typename T>
constexpr int kFull = 16 / static_cast<int>(sizeof(T));

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p) {
    return *reinterpret_cast<const Vec<T, N>*>(p);
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& v) {
    *reinterpret_cast<Vec<T, N>*>(p) = v;
}

// N parameters (a norm's weight or bias) from column c on, kept in 32 bits or
// in the rows' type.
template <typename T, int N>
__device__ __forceinline__ void load_param(float (&out)[N], const void* p, bool f32, int64_t c) {
    if (f32) {
        constexpr int M = N < 4 ? N : 4;  // 16 bytes
#pragma unroll
        for (int i = 0; i < N; i += M) {
            const Vec<float, M> v = load_vec<float, M>(static_cast<const float*>(p) + c + i);
#pragma unroll
            for (int u = 0; u < M; ++u) out[i + u] = v.v[u];
        }
    } else {
        const Vec<T, N> v = load_vec<T, N>(static_cast<const T*>(p) + c);
#pragma unroll
        for (int u = 0; u < N; ++u) out[u] = to_f32(v.v[u]);
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

// CTAs of the backward pass that own partial column sums: four on each of
// 152 SMs.
constexpr int kNormMaxPartials = 608;

cudaError_t launch_norm(const NormParams& p, int dtype, bool vec, cudaStream_t st);
cudaError_t launch_norm_grad(const NormGradParams& p, int dtype, bool vec, cudaStream_t st);

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

cudaError_t launch_permute(const TokenParams& p, int dtype, bool vec, cudaStream_t st, bool pdl);
cudaError_t launch_unpermute(const TokenParams& p, int dtype, bool vec, cudaStream_t st);
cudaError_t launch_unpermute_grad(const TokenParams& p, int dtype, bool vec, cudaStream_t st);

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
    uint32_t vec;  // every pointer is aligned for wide accesses
};

// A launch's tensors travel in its parameters (at most 32764 bytes).
constexpr int kAdamwMaxTensors = 448;

template <int N>
struct AdamwBatch {
    AdamwTensor t[N];
    const float* grad_scale;
    uint64_t seed;
    float beta1, one_minus_beta1, beta2, one_minus_beta2, decay, step_size, inv_root_bc2, eps;
    uint32_t items;
    int count;
};

static_assert(sizeof(AdamwBatch<kAdamwMaxTensors>) <= 32764, "kernel parameters");

constexpr int64_t kAdamwItem = 4096;  // elements of one work item

cudaError_t launch_adamw(const AdamwBatch<kAdamwMaxTensors>& b, int g_dtype, bool mx, cudaStream_t st);

}  // namespace moe
