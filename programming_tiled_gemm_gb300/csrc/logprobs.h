// Internal interface of the kernels in logprobs.cu (not installed).
#pragma once

#include "internal.h"

namespace gemm_gb300 {

constexpr int kMaxTop = 32;  // alternatives of a row: one lane each

struct LogprobsArgs {
    const void* logits;  // [rows][V], row stride ld
    int64_t ld, rows;
    int V, dtype;
    const int64_t* tokens;  // [rows]; outside 0 .. V - 1: none is given
    float temperature;
    float* logprobs;  // [rows]
    float* entropy;   // [rows] or null
    float* stats;     // [rows][2]: the largest logit m and ln sum exp((z - m) / temperature)
    int top;
    float* top_logprobs;  // [rows][top]
    int64_t* top_tokens;  // [rows][top], -1: none
};
int launch_logprobs(const LogprobsArgs& a, int num_sms, cudaStream_t s, int* launches);

struct LogprobsGradArgs {
    const void* logits;
    int64_t ld, rows;
    int V, dtype;
    const int64_t* tokens;
    float temperature;
    const float* stats;
    const float* entropy;    // [rows], read with dentropy
    const float* dlogprobs;  // [rows] or null
    const float* dentropy;   // [rows] or null
    void* dlogits;           // [rows][V] of the logits' type; may be the logits themselves
    int64_t ldd;
};
int launch_logprobs_grad(const LogprobsGradArgs& a, cudaStream_t s, int* launches);

}  // namespace gemm_gb300
