// Conversions and activations of the linear layers' epilogues.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace gemm_gb300 {

template <bool BF16>
__device__ __forceinline__ uint16_t to_16(float v)
{
    if (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    return __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__device__ __forceinline__ float from_16(uint16_t v)
{
    if (BF16) return __bfloat162float(__ushort_as_bfloat16(v));
    return __half2float(__ushort_as_half(v));
}

// z / (1 + e^-z): e^-z = inf gives -0 for large negative z
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act)
{
    switch (act) {
    case GEMM_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] > 0.f ? v[i] : (v[i] <= 0.f ? 0.f : v[i]);  // NaN stays
        break;
    case GEMM_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.5f * v[i] * (1.f + erff(v[i] * 0.70710678118654752f));
            if (i % 4 == 3) asm volatile("" ::: "memory");  // (not all at once: registers)
        }
        break;
    case GEMM_ACT_GELU_TANH:
        // 0.5 (1 + tanh u) = 1 / (1 + e^-2u)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float u2 = 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]);
            v[i] = __fdividef(v[i], 1.f + __expf(-u2));
        }
        break;
    case GEMM_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = silu(v[i]);
        break;
    default: break;
    }
}

}  // namespace gemm_gb300
