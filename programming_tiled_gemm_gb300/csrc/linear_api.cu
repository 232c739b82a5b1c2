// Host side of the linear-layer and routing entry points of include/gemm.h: argument checks,
// workspaces and the order of the launches.
#include <cstdio>

#include "context.h"
#include "linear.h"
#include "moe.h"

using namespace gemm_gb300;

namespace {

constexpr int64_t kLim32 = 0x7fffffffLL - 1024;  // the kernels index sizes in 32 bits

bool is_16(int dtype) { return dtype == GEMM_BF16 || dtype == GEMM_F16; }
int size_of(int dtype) { return dtype == GEMM_F32 ? 4 : 2; }
bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// A matrix of `rows` rows of `cols` used elements: null or a leading dimension below the
// row's length is refused, unless there is nothing to access.
bool bad_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld)
{
    if (rows == 0 || cols == 0) return false;
    return !p || ld < cols || ld > kLim32;
}

// TMA and 16-byte vector operands: aligned base, row stride a multiple of 16 bytes.
bool bad_rows16(const void* p, int64_t rows, int64_t cols, int64_t ld)
{
    return rows > 0 && cols > 0 && (misaligned(p, 16) || ld % 8 != 0);
}

// Grows the workspace to what the product needs, which *need tells run_product.
int reserve_product(gemm_handle_t h, const LinArgs& a, cudaStream_t s, size_t* need)
{
    *need = linear_partials_bytes(a, h->num_sms, h->opt_tc_chunk);
    return *need == 0 ? GEMM_OK : grow_buffer(h, reinterpret_cast<void**>(&h->lin_partials), &h->lin_partials_bytes, *need, s);
}

int run_product(gemm_handle_t h, const LinArgs& a, size_t need, cudaStream_t s)
{
    LinWorkspace ws;
    ws.partials = need > 0 ? h->lin_partials : nullptr;
    ws.counters = h->lin_counters;
    int n = 0;
    const int stall = !h->opt_test_stall ? 0 : h->opt_test_stall_pair > 0 ? h->opt_test_stall_pair : -1;
    const int rc = launch_linear(a, ws, h->num_sms, h->d_status, h->wait_limit_ns, h->opt_tc_chunk, stall, s, &n);
    h->launches += n;
    return rc;
}

// What gemm_linear and gemm_linear_backward check alike.
int check_shape(int64_t M, int64_t K, int64_t N, int act, int dtype, int64_t groups, const int32_t* offsets)
{
    if (M < 0 || K < 0 || N < 0 || groups < 0) return GEMM_ERR_INVALID_ARG;
    if (act < GEMM_ACT_NONE || act > GEMM_ACT_SWIGLU) return GEMM_ERR_INVALID_ARG;
    if (!is_16(dtype)) return dtype == GEMM_F32 ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_INVALID_ARG;
    if (groups > 0 && !offsets) return GEMM_ERR_INVALID_ARG;
    if (groups > 0 && misaligned(offsets, 4)) return GEMM_ERR_ALIGNMENT;
    if (groups > kMaxGroups || M > kLim32 || K > kLim32 || N > kLim32 / 2) return GEMM_ERR_UNSUPPORTED;
    if (act == GEMM_ACT_SWIGLU && N % 8 != 0) return GEMM_ERR_ALIGNMENT;  // W's up columns start at N
    return GEMM_OK;
}

bool bad_stride(int64_t groups, int64_t K, int64_t ld, int64_t stride)
{
    return groups > 1 && K > 0 && (stride < (K - 1) * ld + 1 || stride > ((int64_t)1 << 38));
}

int linear_impl(gemm_handle_t h, const gemm_linear_args* a, void* stream)
{
    if (!h || !a) return GEMM_ERR_INVALID_ARG;
    int rc = check_shape(a->M, a->K, a->N, a->act, a->dtype, a->groups, a->offsets);
    if (rc != GEMM_OK) return rc;
    if (a->y_dtype != GEMM_F32 && a->y_dtype != a->dtype) return GEMM_ERR_INVALID_ARG;
    const int64_t M = a->M, K = a->K, N = a->N, Nw = a->act == GEMM_ACT_SWIGLU ? 2 * N : N;
    const int64_t G = a->groups > 0 ? a->groups : 1;
    if (bad_matrix(a->X, M, K, a->ldx) || bad_matrix(a->W, K, Nw, a->ldw) || bad_matrix(a->Y, M, N, a->ldy) ||
        (a->R && bad_matrix(a->R, M, N, a->ldr)) || (a->Z && bad_matrix(a->Z, M, Nw, a->ldz)) ||
        bad_stride(G, K, a->ldw, a->w_stride))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GEMM_OK;
    const int ys = size_of(a->y_dtype);
    if (bad_rows16(a->X, M, K, a->ldx) || bad_rows16(a->W, K, Nw, a->ldw) || (G > 1 && K > 0 && a->w_stride % 8 != 0) ||
        misaligned(a->Y, ys) || misaligned(a->R, ys) || misaligned(a->Z, 2) || misaligned(a->bias, 2))
        return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    LinArgs l = {};
    l.mode = kLinFwd;
    l.M = M, l.K = K, l.N = N, l.Nw = Nw;
    l.X = a->X, l.ldx = a->ldx;
    l.W = a->W, l.ldw = a->ldw, l.w_stride = a->w_stride;
    l.bias = a->bias;
    l.R = a->R, l.ldr = a->ldr;
    l.Z = a->Z, l.ldz = a->ldz;
    l.out = a->Y, l.ldo = a->ldy;
    l.act = a->act;
    l.bf16 = a->dtype == GEMM_BF16;
    l.out_f32 = a->y_dtype == GEMM_F32;
    l.G = (int)a->groups;
    l.offsets = a->offsets;
    const bool few = linear_is_few(l);
    glog("gemm_linear %s %lldx%lldx%lld, %lld groups, activation %d: %s kernel", dtype_name(a->dtype), (long long)M,
         (long long)N, (long long)K, (long long)a->groups, a->act, few ? "few-row linear" : "tensor-core linear");
    if (few) {
        int n = 0;
        rc = launch_linear_few(l, h->num_sms, reinterpret_cast<cudaStream_t>(stream), &n);
        h->launches += n;
        return rc;
    }
    size_t need = 0;
    rc = reserve_product(h, l, reinterpret_cast<cudaStream_t>(stream), &need);
    if (rc != GEMM_OK) return rc;
    return run_product(h, l, need, reinterpret_cast<cudaStream_t>(stream));
}

int linear_backward_impl(gemm_handle_t h, const gemm_linear_grad_args* a, void* stream)
{
    if (!h || !a) return GEMM_ERR_INVALID_ARG;
    int rc = check_shape(a->M, a->K, a->N, a->act, a->dtype, a->groups, a->offsets);
    if (rc != GEMM_OK) return rc;
    if (a->dw_dtype != GEMM_F32 && a->dw_dtype != a->dtype) return GEMM_ERR_INVALID_ARG;
    const int64_t M = a->M, K = a->K, N = a->N, Nw = a->act == GEMM_ACT_SWIGLU ? 2 * N : N;
    const int64_t G = a->groups > 0 ? a->groups : 1;
    const bool act = a->act != GEMM_ACT_NONE;
    if (bad_matrix(a->dY, M, N, a->lddy) || (act && bad_matrix(a->Z, M, Nw, a->ldz)) ||
        (a->dX && (bad_matrix(a->W, K, Nw, a->ldw) || bad_stride(G, K, a->ldw, a->w_stride) ||
                   bad_matrix(a->dX, M, K, a->lddx))) ||
        (a->dW && (bad_matrix(a->X, M, K, a->ldx) || bad_matrix(a->dW, K, Nw, a->lddw) ||
                   bad_stride(G, K, a->lddw, a->dw_stride))))
        return GEMM_ERR_INVALID_ARG;
    if (bad_rows16(a->dY, M, N, a->lddy) || (act && bad_rows16(a->Z, M, Nw, a->ldz)) ||
        (a->dX && (bad_rows16(a->W, K, Nw, a->ldw) || (G > 1 && K > 0 && a->w_stride % 8 != 0) ||
                   misaligned(a->dX, 2))) ||
        (a->dW && (bad_rows16(a->X, M, K, a->ldx) || misaligned(a->dW, size_of(a->dw_dtype)))) || misaligned(a->db, 4))
        return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    glog("gemm_linear_backward %s %lldx%lldx%lld, %lld groups, activation %d: dX %d, dW %d, db %d",
         dtype_name(a->dtype), (long long)M, (long long)N, (long long)K, (long long)a->groups, a->act, a->dX != nullptr,
         a->dW != nullptr, a->db != nullptr);
    // dZ and db in one pass over dY and Z
    const void* dZ = a->dY;
    int64_t lddz = a->lddy;
    const bool dx = a->dX && M > 0 && K > 0, dw = a->dW && K > 0 && Nw > 0, products = dx || dw;
    LinArgs l = {};
    l.mode = kLinDx;
    l.M = M, l.K = K, l.N = N, l.Nw = Nw;
    l.X = a->X, l.ldx = a->ldx;
    l.W = a->W, l.ldw = a->ldw, l.w_stride = a->w_stride;
    l.bf16 = a->dtype == GEMM_BF16;
    l.G = (int)a->groups;
    l.offsets = a->offsets;
    LinArgs w = l;
    w.mode = kLinDw;
    w.out = a->dW, w.ldo = a->lddw, w.out_stride = a->dw_stride;
    w.out_f32 = a->dw_dtype == GEMM_F32;
    // the products' workspace first: a call whose workspace cannot grow launches nothing
    size_t need_dx = 0, need_dw = 0;
    if (dx && (rc = reserve_product(h, l, s, &need_dx)) != GEMM_OK) return rc;
    if (dw && (rc = reserve_product(h, w, s, &need_dw)) != GEMM_OK) return rc;
    if (M == 0 && a->db && Nw > 0 && cudaMemsetAsync(a->db, 0, (size_t)G * Nw * sizeof(float), s) != cudaSuccess)
        return GEMM_ERR_CUDA;
    if (M > 0 && N > 0 && ((act && products) || a->db)) {
        LinActArgs e = {};
        e.M = M, e.N = N;
        e.dY = a->dY, e.lddy = a->lddy;
        e.Z = a->Z, e.ldz = a->ldz;
        e.db = a->db;
        e.act = a->act;
        e.bf16 = a->dtype == GEMM_BF16;
        e.G = (int)a->groups;
        e.offsets = a->offsets;
        if (act) {
            lddz = (Nw + 7) / 8 * 8;
            rc = grow_buffer(h, &h->lin_dz, &h->lin_dz_bytes, (size_t)M * lddz * 2, s);
            if (rc != GEMM_OK) return rc;
            dZ = e.dZ = h->lin_dz;
            e.lddz = lddz;
        }
        if (a->db) {
            rc = grow_buffer(h, &h->lin_sums, &h->lin_sums_bytes, linear_act_ws_bytes(e, h->num_sms), s);
            if (rc != GEMM_OK) return rc;
        }
        int n = 0;
        if (a->db && dx) {
            l.db_piece = linear_act_piece(e, h->num_sms);
            if (linear_adds_db(l, l.db_piece, h->num_sms, h->opt_tc_chunk)) {
                l.db = a->db;
                l.db_ws = static_cast<float*>(h->lin_sums);
            }
        }
        rc = launch_linear_act(e, static_cast<float*>(h->lin_sums), l.db != nullptr, h->num_sms, s, &n);
        h->launches += n;
        if (rc != GEMM_OK) return rc;
    }
    l.dZ = w.dZ = dZ, l.lddz = w.lddz = lddz;
    if (dx) {
        l.out = a->dX, l.ldo = a->lddx;
        if ((rc = run_product(h, l, need_dx, s)) != GEMM_OK) return rc;
    }
    return dw ? run_product(h, w, need_dw, s) : GEMM_OK;
}

bool known_dtype(int d) { return d == GEMM_F32 || is_16(d); }

int check_routing(int64_t T, int64_t k)
{
    if (T < 0 || k < 1) return GEMM_ERR_INVALID_ARG;
    if (k > kMaxTopK || T > kLim32 / k) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

int route_impl(gemm_handle_t h, int64_t T, int64_t E, int64_t k, const void* logits, int64_t ldl, int dtype,
               int renormalize, float* weights, int32_t* experts, int32_t* slots, int32_t* rows, int32_t* offsets,
               void* stream)
{
    if (!h || E < 1 || k > E || !known_dtype(dtype) || !offsets) return GEMM_ERR_INVALID_ARG;
    int rc = check_routing(T, k);
    if (rc != GEMM_OK) return rc;
    if (E > kMaxExperts) return GEMM_ERR_UNSUPPORTED;
    if (bad_matrix(logits, T, E, ldl) || (T > 0 && (!weights || !experts || !slots || !rows))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, size_of(dtype)) || misaligned(weights, 4) || misaligned(experts, 4) || misaligned(slots, 4) ||
        misaligned(rows, 4) || misaligned(offsets, 4))
        return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return from_cuda(cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, s));
    RouteArgs a = {logits, ldl, T, E, (int)k, dtype, renormalize != 0, weights, experts, slots, rows, offsets};
    rc = grow_buffer(h, &h->route_counts, &h->route_counts_bytes, moe_route_ws_bytes(a, h->num_sms), s);
    if (rc != GEMM_OK) return rc;
    int n = 0;
    rc = launch_moe_route(a, static_cast<int*>(h->route_counts), h->lin_counters + linear_counters(h->num_sms), h->num_sms,
                          s, &n);
    h->launches += n;
    return rc;
}

int route_backward_impl(gemm_handle_t h, int64_t T, int64_t E, int64_t k, const float* dweights, const void* logits,
                        int64_t ldl, int dtype, const int32_t* experts, int renormalize, void* dlogits, int64_t lddl,
                        void* stream)
{
    if (!h || E < 1 || k > E || !known_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
    const int rc = check_routing(T, k);
    if (rc != GEMM_OK) return rc;
    if (E > kMaxExperts) return GEMM_ERR_UNSUPPORTED;
    if (bad_matrix(logits, T, E, ldl) || bad_matrix(dlogits, T, E, lddl) || (T > 0 && (!dweights || !experts)))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, size_of(dtype)) || misaligned(dlogits, size_of(dtype)) || misaligned(dweights, 4) ||
        misaligned(experts, 4))
        return GEMM_ERR_ALIGNMENT;
    if (T == 0) return GEMM_OK;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    RouteGradArgs a = {dweights, logits, ldl, T, E, experts, (int)k, dtype, renormalize != 0, dlogits, lddl};
    int n = 0;
    const int rc2 = launch_moe_route_grad(a, reinterpret_cast<cudaStream_t>(stream), &n);
    h->launches += n;
    return rc2;
}

// What the exchange's entry points check alike.
int check_exchange(gemm_handle_t h, int64_t T, int64_t N, int64_t k, int dtype)
{
    if (!h || N < 0 || !known_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
    const int rc = check_routing(T, k);
    if (rc != GEMM_OK) return rc;
    return N > (1 << 30) ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

int dispatch_impl(gemm_handle_t h, int64_t T, int64_t N, int64_t k, const void* x, int64_t ldx, int dtype,
                  const int32_t* rows, void* xr, int64_t ldxr, void* stream)
{
    const int rc = check_exchange(h, T, N, k, dtype);
    if (rc != GEMM_OK) return rc;
    if (bad_matrix(x, T, N, ldx) || bad_matrix(xr, T, N, ldxr) || (T > 0 && !rows)) return GEMM_ERR_INVALID_ARG;
    if (misaligned(x, size_of(dtype)) || misaligned(xr, size_of(dtype)) || misaligned(rows, 4)) return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    DispatchArgs a = {x, ldx, rows, T, (int)N, (int)k, xr, ldxr};
    int n = 0;
    const int rc2 = launch_moe_dispatch(a, dtype, reinterpret_cast<cudaStream_t>(stream), &n);
    h->launches += n;
    return rc2;
}

int combine_impl(gemm_handle_t h, int64_t T, int64_t N, int64_t k, const void* y, int64_t ldy, int64_t rows_y,
                 int dtype, const int32_t* slots, const float* weights, const void* R, int64_t ldr, void* out,
                 int64_t ldo, void* stream)
{
    const int rc = check_exchange(h, T, N, k, dtype);
    if (rc != GEMM_OK) return rc;
    if (rows_y < 0 || rows_y > kLim32 || bad_matrix(y, rows_y, N, ldy) || (R && bad_matrix(R, T, N, ldr)) ||
        bad_matrix(out, T, N, ldo) || (T > 0 && !slots))
        return GEMM_ERR_INVALID_ARG;
    const int es = size_of(dtype);
    if (misaligned(y, es) || misaligned(R, es) || misaligned(out, es) || misaligned(slots, 4) || misaligned(weights, 4))
        return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    CombineArgs a = {y, ldy, rows_y, slots, weights, R, ldr, T, (int)N, (int)k, out, ldo};
    int n = 0;
    const int rc2 = launch_moe_combine(a, dtype, reinterpret_cast<cudaStream_t>(stream), &n);
    h->launches += n;
    return rc2;
}

int combine_backward_impl(gemm_handle_t h, int64_t T, int64_t N, int64_t k, const void* dout, int64_t lddo,
                          const void* y, int64_t ldy, int dtype, const int32_t* slots, const int32_t* rows,
                          const float* weights, void* dy, int64_t lddy, float* dweights, void* stream)
{
    const int rc = check_exchange(h, T, N, k, dtype);
    if (rc != GEMM_OK) return rc;
    if (bad_matrix(dout, T, N, lddo) || bad_matrix(y, T, N, ldy) || bad_matrix(dy, T, N, lddy) ||
        (T > 0 && (!slots || !rows || !weights || !dweights)))
        return GEMM_ERR_INVALID_ARG;
    const int es = size_of(dtype);
    if (misaligned(dout, es) || misaligned(y, es) || misaligned(dy, es) || misaligned(slots, 4) || misaligned(rows, 4) ||
        misaligned(weights, 4) || misaligned(dweights, 4))
        return GEMM_ERR_ALIGNMENT;
    DeviceGuard g(h->device);
    if (!g.ok()) return GEMM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0 && N == 0) return from_cuda(cudaMemsetAsync(dweights, 0, (size_t)T * k * sizeof(float), s));
    CombineGradArgs a = {dout, lddo, y, ldy, slots, rows, weights, T, (int)N, (int)k, dy, lddy, dweights};
    int n = 0;
    const int rc2 = launch_moe_combine_grad(a, dtype, s, &n);
    h->launches += n;
    return rc2;
}

int told(const char* what, int rc)
{
    if (rc != GEMM_OK) glog("%s refused: %s (%d)", what, gemm_status_string(rc), rc);
    return rc;
}

}  // namespace

extern "C" {

int gemm_linear(gemm_handle_t h, const gemm_linear_args* args, void* stream)
{
    return told("gemm_linear", linear_impl(h, args, stream));
}

int gemm_linear_backward(gemm_handle_t h, const gemm_linear_grad_args* args, void* stream)
{
    return told("gemm_linear_backward", linear_backward_impl(h, args, stream));
}

int moe_route(gemm_handle_t h, int64_t T, int64_t E, int64_t k, const void* logits, int64_t ldl, int dtype,
              int renormalize, float* weights, int32_t* experts, int32_t* slots, int32_t* rows, int32_t* offsets,
              void* stream)
{
    return told("moe_route", route_impl(h, T, E, k, logits, ldl, dtype, renormalize, weights, experts, slots, rows,
                                        offsets, stream));
}

int moe_route_backward(gemm_handle_t h, int64_t T, int64_t E, int64_t k, const float* dweights, const void* logits,
                       int64_t ldl, int dtype, const int32_t* experts, int renormalize, void* dlogits, int64_t lddl,
                       void* stream)
{
    return told("moe_route_backward", route_backward_impl(h, T, E, k, dweights, logits, ldl, dtype, experts,
                                                          renormalize, dlogits, lddl, stream));
}

int moe_dispatch(gemm_handle_t h, int64_t T, int64_t N, int64_t k, const void* x, int64_t ldx, int dtype,
                 const int32_t* rows, void* xr, int64_t ldxr, void* stream)
{
    return told("moe_dispatch", dispatch_impl(h, T, N, k, x, ldx, dtype, rows, xr, ldxr, stream));
}

int moe_combine(gemm_handle_t h, int64_t T, int64_t N, int64_t k, const void* y, int64_t ldy, int64_t rows_y,
                int dtype, const int32_t* slots, const float* weights, const void* R, int64_t ldr, void* out,
                int64_t ldo, void* stream)
{
    return told("moe_combine", combine_impl(h, T, N, k, y, ldy, rows_y, dtype, slots, weights, R, ldr, out, ldo,
                                            stream));
}

int moe_combine_backward(gemm_handle_t h, int64_t T, int64_t N, int64_t k, const void* dout, int64_t lddo,
                         const void* y, int64_t ldy, int dtype, const int32_t* slots, const int32_t* rows,
                         const float* weights, void* dy, int64_t lddy, float* dweights, void* stream)
{
    return told("moe_combine_backward", combine_backward_impl(h, T, N, k, dout, lddo, y, ldy, dtype, slots, rows,
                                                              weights, dy, lddy, dweights, stream));
}

}  // extern "C"
