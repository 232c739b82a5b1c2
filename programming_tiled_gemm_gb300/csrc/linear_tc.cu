// Linear layers on the tensor cores: the choice among the kernel's variants (the kernel itself is in
// linear_pair.h) and their launches.
#include "linear.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(linear_tc)

}  // namespace gemm_gb300

#include "linear_pair.h"

namespace gemm_gb300 {

namespace {

template <bool BF16, bool CHUNKED>
int launch_typed(int mode, const LinPlan& pl, const CUtensorMap& tmA, const CUtensorMap& tmB, const LinParams& p,
                 int num_sms, cudaStream_t s)
{
    if (mode == kLinDw) return launch_plain<kLinDw, false, BF16, CHUNKED, 1>(pl, tmA, tmB, p, num_sms, s);
    if constexpr (!CHUNKED) {  // (chunked tiles are narrow)
        if (pl.kps == 1) {
            if (mode == kLinDx) return launch_plain<kLinDx, false, BF16, false, 1>(pl, tmA, tmB, p, num_sms, s);
            if (pl.gated) return launch_plain<kLinFwd, true, BF16, false, 1>(pl, tmA, tmB, p, num_sms, s);
            return launch_plain<kLinFwd, false, BF16, false, 1>(pl, tmA, tmB, p, num_sms, s);
        }
    }
    if (mode == kLinDx) return launch_plain<kLinDx, false, BF16, CHUNKED, 2>(pl, tmA, tmB, p, num_sms, s);
    if (pl.gated) return launch_plain<kLinFwd, true, BF16, CHUNKED, 2>(pl, tmA, tmB, p, num_sms, s);
    return launch_plain<kLinFwd, false, BF16, CHUNKED, 2>(pl, tmA, tmB, p, num_sms, s);
}

}  // namespace

// One warp a CTA has some 1500 cycles a round of loads; a launch of its own takes 8000 (4 us).
bool linear_adds_db(const LinArgs& a, int piece, int num_sms, int kc)
{
    const LinPlan pl = plan(a, num_sms, is_chunked(a, kc));
    const int64_t G = a.G > 0 ? a.G : 1, items = G * ((a.Nw + 31) / 32);
    const int64_t ctas = 2 * (pl.tiles < pl.pairs ? pl.tiles : (int64_t)pl.pairs);
    if (ctas < 1 || items > (1 << 30)) return false;
    const int64_t pieces = a.M / G / piece + 1;  // of a group, on average
    const double sums = 1500. * (double)((items + ctas - 1) / ctas) * (double)((pieces + 15) / 16);
    const double tiles = (double)((pl.tiles + pl.pairs - 1) / pl.pairs) * pl.kb * kb_cycles(pl.wmax);
    return sums <= tiles + 8000.;
}

size_t linear_partials_bytes(const LinArgs& a, int num_sms, int kc)
{
    const LinPlan pl = plan(a, num_sms, is_chunked(a, kc));
    if (pl.split_w == 0) return 0;
    return (size_t)pl.pairs * 2 * CTA_F * pl.wmax * sizeof(float);
}

int64_t linear_counters(int num_sms) { return num_sms; }  // two a tile of the last wave, fewer tiles than pairs

int launch_linear(const LinArgs& a, const LinWorkspace& ws, int num_sms, int* dev_status, uint64_t limit_ns, int kc,
                  int test_stall, cudaStream_t stream, int* launches)
{
    const bool chunked = is_chunked(a, kc);
    const LinPlan pl = plan(a, num_sms, chunked);
    if (pl.tiles <= 0) return GEMM_OK;
    LinParams p;
    CUtensorMap tmA, tmB;
    const int ready = set_up(a, pl, ws, dev_status, limit_ns, kc, test_stall, p, tmA, tmB);
    if (ready != GEMM_OK) return ready;
    const auto launch = a.bf16 ? (chunked ? launch_typed<true, true> : launch_typed<true, false>)
                               : (chunked ? launch_typed<false, true> : launch_typed<false, false>);
    const int rc = launch(a.mode, pl, tmA, tmB, p, num_sms, stream);
    if (rc == GEMM_OK) *launches += 1;
    return rc;
}

}  // namespace gemm_gb300
