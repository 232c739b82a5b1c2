// Host side of the entry points of include/gemm.h that stand around the linear layers of a model
// in use: argument checks, workspaces and the order of the launches.
#include <cmath>

#include "api_checks.h"
#include "context.h"
#include "linear.h"
#include "logprobs.h"
#include "moe.h"

using namespace gemm_gb300;

namespace {

bool bad_stride(int64_t E, int64_t rows, int64_t cols, int64_t ld, int64_t stride)
{
    return E > 1 && (stride < (rows - 1) * ld + cols || stride > ((int64_t)1 << 38));
}

int layer_impl(gemm_handle_t h, const moe_layer_args* a, void* stream)
{
    if (!h || !a) return GEMM_ERR_INVALID_ARG;
    const int64_t T = a->T, E = a->E, k = a->k, D = a->D, F = a->F;
    if (T < 0 || E < 1 || k < 1 || k > E || D < 0 || F < 1) return GEMM_ERR_INVALID_ARG;
    if (a->act < GEMM_ACT_NONE || a->act > GEMM_ACT_SWIGLU || !known_dtype(a->logits_dtype)) return GEMM_ERR_INVALID_ARG;
    if (!is_16(a->dtype)) return a->dtype == GEMM_F32 ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_INVALID_ARG;
    if (a->y_dtype != GEMM_F32 && a->y_dtype != a->dtype) return GEMM_ERR_INVALID_ARG;
    if (T > kLayerTokens || k > kMaxTopK || E > kMaxExperts || D > (int64_t)kLayerSlab * kLayerCounters || F > (1 << 24))
        return GEMM_ERR_UNSUPPORTED;
    const int64_t Fw = a->act == GEMM_ACT_SWIGLU ? 2 * F : F;
    if (bad_matrix(a->logits, T, E, a->ldl) || bad_matrix(a->X, T, D, a->ldx) || bad_matrix(a->W1, D, Fw, a->ldw1) ||
        bad_matrix(a->W2, F, D, a->ldw2) || (a->R && bad_matrix(a->R, T, D, a->ldr)) || bad_matrix(a->Y, T, D, a->ldy) ||
        (D > 0 && (bad_stride(E, D, Fw, a->ldw1, a->w1_stride) || bad_stride(E, F, D, a->ldw2, a->w2_stride))))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return GEMM_OK;
    const int ys = size_of(a->y_dtype);
    if (bad_rows16(a->X, T, D, a->ldx) || bad_rows16(a->W1, D, Fw, a->ldw1) || bad_rows16(a->W2, F, D, a->ldw2) ||
        (E > 1 && (a->w1_stride % 8 != 0 || a->w2_stride % 8 != 0)) || (a->act == GEMM_ACT_SWIGLU && F % 8 != 0) ||
        misaligned(a->logits, size_of(a->logits_dtype)) || misaligned(a->b1, 2) || misaligned(a->b2, 2) ||
        misaligned(a->R, ys) || misaligned(a->Y, ys))
        return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    glog("moe_layer %s, %lld tokens to %lld of %lld experts, %lld -> %lld, activation %d", dtype_name(a->dtype), (long long)T,
         (long long)k, (long long)E, (long long)D, (long long)F, a->act);
    LayerArgs l = {};
    l.T = (int)T, l.E = (int)E, l.k = (int)k, l.D = (int)D, l.F = (int)F, l.Fw = (int)Fw;
    l.logits = a->logits, l.ldl = a->ldl, l.logits_dtype = a->logits_dtype, l.renormalize = a->renormalize != 0;
    l.x = a->X, l.ldx = a->ldx;
    l.w1 = a->W1, l.ldw1 = a->ldw1, l.w1_stride = a->w1_stride, l.b1 = a->b1;
    l.w2 = a->W2, l.ldw2 = a->ldw2, l.w2_stride = a->w2_stride, l.b2 = a->b2;
    l.R = a->R, l.ldr = a->ldr;
    l.out = a->Y, l.ldo = a->ldy;
    l.act = a->act, l.bf16 = a->dtype == GEMM_BF16, l.out_f32 = a->y_dtype == GEMM_F32;
    int rc = grow_buffer(h, &h->layer, &h->layer_bytes, moe_layer_ws_bytes(l), s);
    if (rc != GEMM_OK) return rc;
    int n = 0;
    rc = launch_moe_layer(l, h->layer, h->lin_counters + linear_counters(h->num_sms) + 1, h->num_sms, h->d_status,
                          h->wait_limit_ns, h->opt_test_stall, s, &n);
    h->launches += n;
    return rc;
}

// What token_logprobs and token_logprobs_backward check alike.
int check_logprobs(gemm_handle_t h, int64_t rows, int64_t V, const void* logits, int64_t ld, int dtype,
                   const int64_t* tokens, float temperature, const float* stats)
{
    if (!h || rows < 0 || V < 1 || !known_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
    // (the kernels multiply by 1 / (T ln 2), which is infinite before 1 / T is)
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite((float)(1.4426950408889634 / temperature)))
        return GEMM_ERR_INVALID_ARG;
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

int moe_layer(gemm_handle_t h, const moe_layer_args* args, void* stream)
{
    return told("moe_layer", layer_impl(h, args, stream));
}

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
