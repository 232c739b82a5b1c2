// Host side of the entry points of include/gemm.h that stand around the linear layers of a model
// in use: argument checks, workspaces and the order of the launches.
#include <cmath>

#include "api_checks.h"
#include "context.h"
#include "logprobs.h"

using namespace gemm_gb300;

namespace {

// What token_logprobs and token_logprobs_backward check alike.
int check_logprobs(gemm_handle_t h, int64_t rows, int64_t V, const void* logits, int64_t ld, int dtype,
                   const int64_t* tokens, float temperature, const float* stats)
{
    if (!h || rows < 0 || V < 1 || !known_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature)) return GEMM_ERR_INVALID_ARG;
    if (V > (1 << 30) || rows > kLim32) return GEMM_ERR_UNSUPPORTED;
    if (bad_matrix(logits, rows, V, ld) || (rows > 0 && (!tokens || !stats))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, size_of(dtype)) || misaligned(tokens, 8) || misaligned(stats, 4)) return GEMM_ERR_ALIGNMENT;
    return GEMM_OK;
}

int logprobs_impl(gemm_handle_t h, int64_t rows, int64_t V, const void* logits, int64_t ld, int dtype,
                  const int64_t* tokens, float temperature, float* logprobs, float* entropy, float* stats, int64_t top,
                  float* top_logprobs, int64_t* top_tokens, void* stream)
{
    const int rc = check_logprobs(h, rows, V, logits, ld, dtype, tokens, temperature, stats);
    if (rc != GEMM_OK) return rc;
    if (top < 0 || (rows > 0 && (!logprobs || (top > 0 && (!top_logprobs || !top_tokens))))) return GEMM_ERR_INVALID_ARG;
    if (top > kMaxTop) return GEMM_ERR_UNSUPPORTED;
    if (misaligned(logprobs, 4) || misaligned(entropy, 4) || (top > 0 && (misaligned(top_logprobs, 4) || misaligned(top_tokens, 8))))
        return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    glog("token_logprobs %s %lldx%lld, entropy %d, %lld alternatives", dtype_name(dtype), (long long)rows, (long long)V,
         entropy != nullptr, (long long)top);
    LogprobsArgs a = {logits, ld, rows, (int)V, dtype, tokens, temperature, logprobs, entropy, stats, (int)top,
                      top_logprobs, top_tokens};
    int n = 0;
    const int rc2 = launch_logprobs(a, h->num_sms, reinterpret_cast<cudaStream_t>(stream), &n);
    h->launches += n;
    return rc2;
}

int logprobs_backward_impl(gemm_handle_t h, int64_t rows, int64_t V, const void* logits, int64_t ld, int dtype,
                           const int64_t* tokens, float temperature, const float* stats, const float* entropy,
                           const float* dlogprobs, const float* dentropy, void* dlogits, int64_t ldd, void* stream)
{
    const int rc = check_logprobs(h, rows, V, logits, ld, dtype, tokens, temperature, stats);
    if (rc != GEMM_OK) return rc;
    if (bad_matrix(dlogits, rows, V, ldd) || (dentropy && !entropy)) return GEMM_ERR_INVALID_ARG;
    if (dlogits == logits && ldd != ld && rows > 1) return GEMM_ERR_INVALID_ARG;
    if (misaligned(entropy, 4) || misaligned(dlogprobs, 4) || misaligned(dentropy, 4) || misaligned(dlogits, size_of(dtype)))
        return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    LogprobsGradArgs a = {logits, ld, rows, (int)V, dtype, tokens, temperature, stats, entropy, dlogprobs, dentropy,
                          dlogits, ldd};
    int n = 0;
    const int rc2 = launch_logprobs_grad(a, reinterpret_cast<cudaStream_t>(stream), &n);
    h->launches += n;
    return rc2;
}

}  // namespace

extern "C" {

int token_logprobs(gemm_handle_t h, int64_t rows, int64_t V, const void* logits, int64_t ld, int dtype,
                   const int64_t* tokens, float temperature, float* logprobs, float* entropy, float* stats,
                   int64_t top, float* top_logprobs, int64_t* top_tokens, void* stream)
{
    return told("token_logprobs", logprobs_impl(h, rows, V, logits, ld, dtype, tokens, temperature, logprobs, entropy,
                                                stats, top, top_logprobs, top_tokens, stream));
}

int token_logprobs_backward(gemm_handle_t h, int64_t rows, int64_t V, const void* logits, int64_t ld, int dtype,
                            const int64_t* tokens, float temperature, const float* stats, const float* entropy,
                            const float* dlogprobs, const float* dentropy, void* dlogits, int64_t ldd, void* stream)
{
    return told("token_logprobs_backward", logprobs_backward_impl(h, rows, V, logits, ld, dtype, tokens, temperature, stats,
                                                                  entropy, dlogprobs, dentropy, dlogits, ldd, stream));
}

}  // extern "C"
