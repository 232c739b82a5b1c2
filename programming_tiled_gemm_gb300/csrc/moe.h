// Internal interface of the mixture-of-experts kernels in moe.cu (not installed).
#pragma once

#include "internal.h"

namespace gemm_gb300 {

constexpr int kMaxExperts = 1024;  // logits of a token in a warp's registers
constexpr int kMaxTopK = 32;       // one lane a pick

// Larger values have larger keys; NaN (as the largest) before +inf, 0 for -inf.  +0 = -0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// The value of a key (a NaN for any NaN's).
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

struct RouteArgs {
    const void* logits;  // [T][E], row stride ld
    int64_t ld, T, E;
    int k, dtype, renormalize;
    float* weights;  // [T][k]
    int* experts;    // [T][k], -1: none
    int* slots;      // [T][k]: place in the order by expert, -1: none
    int* rows;       // [T k]: the assignment t k + j at each place, -1 past the last
    int* offsets;    // [E + 1]
};
size_t moe_route_ws_bytes(const RouteArgs& a, int num_sms);
// `counter` is zero before and after every launch.  Returns a gemm_status_t.
int launch_moe_route(const RouteArgs& a, int* ws, unsigned* counter, int num_sms, cudaStream_t s, int* launches);

struct RouteGradArgs {
    const float* dweights;  // [T][k]
    const void* logits;
    int64_t ld, T, E;
    const int* experts;
    int k, dtype, renormalize;
    void* dlogits;  // [T][E] of the logits' type
    int64_t ldd;
};
int launch_moe_route_grad(const RouteGradArgs& a, cudaStream_t s, int* launches);

struct DispatchArgs {
    const void* x;  // [T][N]
    int64_t ldx;
    const int* rows;
    int64_t T;
    int N, k;
    void* xr;  // [T k][N]
    int64_t ldxr;
};
int launch_moe_dispatch(const DispatchArgs& a, int dtype, cudaStream_t s, int* launches);

struct CombineArgs {
    const void* y;  // [rows_y][N]
    int64_t ldy, rows_y;
    const int* slots;
    const float* weights;  // [T][k] or null: ones
    const void* R;         // [T][N] or null
    int64_t ldr, T;
    int N, k;
    void* out;  // [T][N]
    int64_t ldo;
};
int launch_moe_combine(const CombineArgs& a, int dtype, cudaStream_t s, int* launches);

struct CombineGradArgs {
    const void* dout;  // [T][N]
    int64_t lddo;
    const void* y;  // [T k][N]
    int64_t ldy;
    const int* slots;
    const int* rows;
    const float* weights;
    int64_t T;
    int N, k;
    void* dy;  // [T k][N]
    int64_t lddy;
    float* dweights;  // [T][k]
};
int launch_moe_combine_grad(const CombineGradArgs& a, int dtype, cudaStream_t s, int* launches);

// A whole layer for a few tokens (moe_layer.cu).
constexpr int kLayerTokens = 64;
constexpr int kLayerSlab = 64;       // columns of W2 that one counter stands for
constexpr int kLayerCounters = 4096;  // and the counters there are, zero before and after every launch

struct LayerArgs {
    int T, E, k, D, F, Fw;  // Fw columns of W1 (2 F when gated)
    const void* logits;     // [T][E] of type logits_dtype
    int64_t ldl;
    int logits_dtype, renormalize;
    const void* x;  // [T][D]
    int64_t ldx;
    const void* w1;  // [E][D][Fw]
    int64_t ldw1, w1_stride;
    const void* b1;  // [E][Fw] or null
    const void* w2;  // [E][F][D]
    int64_t ldw2, w2_stride;
    const void* b2;  // [E][D] or null
    const void* R;   // [T][D] or null
    int64_t ldr;
    void* out;  // [T][D]
    int64_t ldo;
    int act;
    bool bf16, out_f32;
};
size_t moe_layer_ws_bytes(const LayerArgs& a);
int launch_moe_layer(const LayerArgs& a, void* ws, unsigned* counters, int num_sms, int* dev_status, uint64_t limit_ns,
                     int test_stall, cudaStream_t s, int* launches);

}  // namespace gemm_gb300
