// The forward product with low-rank adapters on the tensor cores: linear_pair.h's kernel with a longer
// reduction, and its launches.
#include "linear.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(linear_adapted)

}  // namespace gemm_gb300

#include "linear_pair.h"

namespace gemm_gb300 {

namespace {

template <bool GATED, bool BF16, int KPS>
__global__ void __launch_bounds__(THREADS, 1)
linear_adapted_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmE, LinParams p, AdaptParams ad)
{
    linear_pair_body<kLinFwd, GATED, BF16, false, KPS, true>(tmA, tmB, tmE, p, ad);
}

template <bool GATED, bool BF16, int KPS>
int launch_typed(const LinPlan& pl, const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmE,
                 const LinParams& p, const AdaptParams& ad, int num_sms, cudaStream_t stream)
{
    static std::atomic<int> fit{0};
    static std::atomic<uint64_t> allowed{0};
    return launch_kernel(linear_adapted_kernel<GATED, BF16, KPS>, fit, allowed, pl, p.split_w, num_sms, stream, tmA, tmB, tmE,
                         p, ad);
}

}  // namespace

int linear_tile_rows(const LinArgs& a, int num_sms)
{
    const LinPlan pl = plan(a, num_sms, false);
    return tile_width(kLinFwd, pl.rows, pl.wcap);
}

int launch_linear_adapted(const LinArgs& a, const LinWorkspace& ws, int num_sms, int* dev_status, uint64_t limit_ns,
                          int test_stall, cudaStream_t stream, int* launches)
{
    if (is_chunked(a, 0) || !a.adapt || a.G != 0) return GEMM_ERR_UNSUPPORTED;
    const LinAdapt& l = *a.adapt;
    const LinPlan pl = plan(a, num_sms, false);
    if (pl.tiles <= 0) return GEMM_OK;
    LinParams p;
    CUtensorMap tmA, tmB, tmE = {};
    int rc = set_up(a, pl, ws, dev_status, limit_ns, 0, test_stall, p, tmA, tmB);
    if (rc != GEMM_OK) return rc;
    AdaptParams ad = {l.u, l.tiles, l.slot, l.bad, l.rs, l.n, adapter_list_words(l.tile_rows), pl.places};
    if (!encode(&tmE, 3, l.B, a.bf16, a.Nw, l.r, l.n, l.ldb, l.n > 1 ? l.b_stride : l.ldb, l.rs < BK ? l.rs : BK))
        return GEMM_ERR_CUDA;
    const auto launch = pl.gated ? (a.bf16 ? (pl.kps == 1 ? launch_typed<true, true, 1> : launch_typed<true, true, 2>)
                                           : (pl.kps == 1 ? launch_typed<true, false, 1> : launch_typed<true, false, 2>))
                                 : (a.bf16 ? (pl.kps == 1 ? launch_typed<false, true, 1> : launch_typed<false, true, 2>)
                                           : (pl.kps == 1 ? launch_typed<false, false, 1> : launch_typed<false, false, 2>));
    rc = launch(pl, tmA, tmB, tmE, p, ad, num_sms, stream);
    if (rc == GEMM_OK) *launches += 1;
    return rc;
}

}  // namespace gemm_gb300
