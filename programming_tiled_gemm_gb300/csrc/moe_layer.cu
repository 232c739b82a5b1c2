// A whole mixture-of-experts layer for up to 64 tokens, in two kernels:
//   out[t] = sum_j w[t][j] (act(x[t] W1[e] + b1[e]) W2[e] + b2[e]) + R[t],   e = e[t][j], the router's picks.
//
// Bound by the picked experts' weights, which are streamed once: 64 tokens are too few rows to keep
// the tensor cores busy.  Each kernel's CTAs walk (expert, 64 columns of its matrix) items; one warp
// keeps a ring of stages filled across the items, 128 of the reduced dimension a stage: the weights by
// TMA, the expert's rows by 16-byte copies.  Eight warps multiply with mma.sync: the features on the M
// side, eight rows an MMA on the N side, so that a single row costs one MMA of 16 x 16 weights.
// (tcgen05's set-up, tile of 128 features and drain take longer than such an item; FMAs would bound
// three rows and more.)
//
// Every CTA routes for itself: the picks are some hundred instructions of a warp a token, less than
// a launch and a trip through memory.  A pick's row of H and of the partial outputs is its index
// t k + j, so nothing is sorted and CTAs need not agree on more than that; an expert's rows are the
// picks that name it, in order.  The second kernel is launched early, routes and fills its ring with
// weights while the first one ends, and waits for it only before it reads H.  It leaves every pick's
// product in fp32; the CTA that finishes a slab of columns last adds each token's picks in the order
// of j, the residual last.  Nothing waits for another CTA, and no sum depends on their order.
//
// Measured (bf16, swiglu, GPU time): 1 token to 4 of 64 experts, 2048 -> 1024 -> 2048, 19.8 us (50 MB, floor 7.4:
// routing, first copies, the kernels' hand-over and the slabs' sums each take 1 to 4); 16 tokens 98 us (519 MB, 5.3
// TB/s in all, 6.2 in the first kernel's loop); 64 tokens to 2 of 16, 4096 -> 4096 -> 4096, 280 to 287 us (1.6 GB, 5.7 TB/s;
// DRAM 79 % busy in the first kernel).
// Dropped: one warp for the weights' and the rows' copies (64 tokens: 330 us instead of 290); every warp at every stage
// (476 instead of 332 then); weights by cp.async from all threads, a block barrier a stage (16 tokens: 184 instead of 103);
// the second kernel's last round of items cut along its reduced dimension (64 tokens 292 instead of 280, one token 23).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear.h"
#include "linear_math.h"
#include "moe.h"
#include "ptx.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(moe_layer)

namespace {

constexpr int MMA_WARPS = 8, WARPS = MMA_WARPS + 2, THREADS = 32 * WARPS;  // the last two load weights and rows
constexpr int SLAB = kLayerSlab;  // columns of W an item
constexpr int DEPTH = 128;        // of the reduced dimension a stage
// Stages after which the sums are put aside, 4096 of the reduced dimension: an MMA truncates what it adds to, so that a
// sum of one sign loses in proportion to its length (1.2e-5 of the result at F 16384, 3.9e-4 at 262144; with this 1.7e-6 at
// either, and 8 experts of 4096 x 14336 take 444 us for 32 tokens instead of 437, 1 to 8 of 4096 x 4096 0.5 % more).
constexpr int RESTART = 4096 / DEPTH;
constexpr int W_BYTES = DEPTH * SLAB * 2;
constexpr int ROW_BYTES = DEPTH * 2 + 16;  // of X or H a stage: rows 16 bytes apart in the banks
constexpr int MAX_STAGES = 8;  // (an even number of them: each belongs to one half of the warps, which sees its every phase)
constexpr int SMEM_TWO = 112 * 1024, SMEM_ONE = 224 * 1024;  // of a CTA, two or one an SM
constexpr int PAD = SLAB + 4;         // floats of a row of sums
constexpr int MAX_ROWS = 32;           // of an item: an expert with more has several
constexpr int MAX_TILES = MAX_ROWS / 8;
constexpr uint16_t NONE = 0xffff;

struct LayerParams {
    int T, E, k, D, F, Fw;
    const void* logits;
    int64_t ldl;
    int logits_dtype, renorm;
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* bias;  // this kernel's
    const void* R;
    int64_t ldr;
    void* out;
    int64_t ldo;
    int act, out_f32;
    uint16_t* h;  // [T k][Fp]
    int Fp;
    float* y;  // [T k][Dp]
    int Dp;
    unsigned* counters;
    int slabs, stages, rows_cap;  // rows_cap: rows of a stage, T to a multiple of 8, or MAX_ROWS
    int* status;
    uint64_t limit_ns;
    int test_stall;
};

// The router's outcome, in shared memory.
struct Routes {
    float* weight;      // [T k]
    uint16_t* expert;   // [T k], NONE: no pick
    uint16_t* pick;     // [T k]: the picks by expert, each expert's in order
    unsigned* tokens;   // [E][2]: a bit a token that picked it
    int* base;          // [E]: its first pick in `pick`
    uint16_t* active;   // [most_groups]: experts with picks, once for each MAX_ROWS of them
    int* first;         // [most_groups + 1]: the groups' first pick in `pick`
    int* n_active;
};
__host__ __device__ inline int most_groups(int picks, int E) { return (E < picks ? E : picks) + picks / MAX_ROWS; }
__host__ __device__ inline int routes_bytes(int picks, int E)
{
    return 16 + 4 * (most_groups(picks, E) + 1) + 12 * E + 4 * picks + 2 * picks * 2 + 2 * most_groups(picks, E) + 16;
}
__device__ __forceinline__ Routes carve(uint8_t* at, int picks, int E)
{
    Routes r;
    r.n_active = reinterpret_cast<int*>(at);
    r.first = r.n_active + 4;
    r.base = r.first + most_groups(picks, E) + 1;
    r.tokens = reinterpret_cast<unsigned*>(r.base + E);
    r.weight = reinterpret_cast<float*>(r.tokens + 2 * E);
    r.expert = reinterpret_cast<uint16_t*>(r.weight + picks);
    r.pick = r.expert + picks;
    r.active = r.pick + picks;
    return r;
}

// (read past L1: the second kernel does so before it has waited for the first)
__device__ __forceinline__ float logit(const LayerParams& p, int t, int e)
{
    const int64_t i = (int64_t)t * p.ldl + e;
    if (p.logits_dtype == GEMM_F32) return __ldcg(static_cast<const float*>(p.logits) + i);
    const uint16_t v = __ldcg(static_cast<const uint16_t*>(p.logits) + i);
    return p.logits_dtype == GEMM_BF16 ? from_16<true>(v) : from_16<false>(v);
}

// One pick: the largest key over the warp, the lowest expert that has it (-1: none is left).
__device__ __forceinline__ int pick_of(uint32_t best, int at, uint32_t& key)
{
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    key = m;
    if (m == 0) return -1;
    const unsigned who = __ballot_sync(0xffffffffu, best == m);
    if (who & (who - 1)) return (int)__reduce_min_sync(0xffffffffu, best == m ? (unsigned)at : 0xffffffffu);
    return __shfl_sync(0xffffffffu, at, __ffs(who) - 1);
}

// What a token's picks leave: its experts, the experts' tokens and, where they are wanted, the weights
// (`all`: a lane's part of the sum over all experts).
template <bool WEIGHTS>
__device__ __forceinline__ void record(const LayerParams& p, const Routes& r, int t, int pick, float val, float top, float all)
{
    const int lane = threadIdx.x % 32, k = p.k;
    if (lane < k) {
        r.expert[t * k + lane] = pick >= 0 ? (uint16_t)pick : NONE;
        if (pick >= 0) atomicOr(&r.tokens[2 * pick + t / 32], 1u << (t % 32));
    }
    if (WEIGHTS) {
        const float ex = pick >= 0 ? expf(val - top) : 0.f;
        float sum = p.renorm ? ex : all;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane < k) r.weight[t * k + lane] = pick >= 0 ? ex / sum : 0.f;
    }
}

// G lanes a token, up to G x REG experts, a lane's keys in registers.  Eight lanes a token are 40 tokens at once.  (48
// tokens to 2 of 16 experts, us of the two kernels: 2.6 and 3.6; a warp a token, one after another, 5.6 and 6.6; four of
// a warp's together 3.6 and 4.9.  One token to 4 of 64: 1.5 and 1.5, with a warp to itself 1.0 and 1.0.)
template <bool WEIGHTS, int G, int REG>
__device__ __forceinline__ void route_few(const LayerParams& p, const Routes& r)
{
    constexpr int PER_WARP = 32 / G;
    const int warp = threadIdx.x / 32, sub = threadIdx.x % 32 / G, lane = threadIdx.x % G, k = p.k;
    for (int t0 = warp * PER_WARP; t0 < p.T; t0 += WARPS * PER_WARP) {
        const int t = t0 + sub;
        const bool live = t < p.T;
        uint32_t key[REG] = {};
        // (all of the loads before the first use)
        const int64_t from = (int64_t)t * p.ldl + lane;
        if (p.logits_dtype == GEMM_F32) {
#pragma unroll
            for (int c = 0; c < REG; ++c)
                if (live && G * c + lane < p.E) key[c] = __ldcg(static_cast<const uint32_t*>(p.logits) + from + G * c);
        } else {
#pragma unroll
            for (int c = 0; c < REG; ++c)
                if (live && G * c + lane < p.E) key[c] = __ldcg(static_cast<const uint16_t*>(p.logits) + from + G * c);
        }
#pragma unroll
        for (int c = 0; c < REG; ++c) {
            const float l = p.logits_dtype == GEMM_F32    ? __uint_as_float(key[c])
                            : p.logits_dtype == GEMM_BF16 ? from_16<true>((uint16_t)key[c])
                                                          : from_16<false>((uint16_t)key[c]);
            key[c] = live && G * c + lane < p.E ? order_key(l) : 0;
        }
        float top = 0.f, sum = 0.f;
        for (int j = 0; j < k; ++j) {
            // the largest key, the lowest expert that has it (0: none is left)
            uint32_t best = key[0];
            int at = lane;
#pragma unroll
            for (int c = 1; c < REG; ++c)
                if (key[c] > best) best = key[c], at = G * c + lane;
#pragma unroll
            for (int d = G / 2; d > 0; d /= 2) {
                const uint32_t o = __shfl_xor_sync(0xffffffffu, best, d);
                const int o_at = __shfl_xor_sync(0xffffffffu, at, d);
                if (o > best || (o == best && o_at < at)) best = o, at = o_at;
            }
            if (WEIGHTS && j == 0) {
                top = best != 0 ? key_value(best) : 0.f;
                if (!p.renorm) {
#pragma unroll
                    for (int c = 0; c < REG; ++c)
                        if (key[c] != 0) sum += expf(key_value(key[c]) - top);
#pragma unroll
                    for (int d = G / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                }
            }
            const float ex = WEIGHTS && best != 0 ? expf(key_value(best) - top) : 0.f;
            if (WEIGHTS && p.renorm) sum += ex;
            if (live && lane == 0) {
                r.expert[t * k + j] = best != 0 ? (uint16_t)at : NONE;
                if (WEIGHTS) r.weight[t * k + j] = ex;
                if (best != 0) atomicOr(&r.tokens[2 * at + t / 32], 1u << (t % 32));
            }
#pragma unroll
            for (int c = 0; c < REG; ++c)
                if (G * c + lane == at) key[c] = 0;
        }
        if (WEIGHTS) {
            __syncwarp();
            if (live)
                for (int j = lane; j < k; j += G)
                    if (r.expert[t * k + j] != NONE) r.weight[t * k + j] /= sum;
        }
    }
}

// The picks of all tokens as moe_route makes them, a warp a token.  Keys of more than 256 experts lie in
// `scratch` (WARPS * E words).
template <bool WEIGHTS>
__device__ __forceinline__ void route(const LayerParams& p, const Routes& r, uint32_t* scratch)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = p.E, k = p.k, picks = p.T * k;
    for (int e = threadIdx.x; e < 2 * E; e += THREADS) r.tokens[e] = 0;
    __syncthreads();
    if (E <= 64) {
        if (p.T <= WARPS) route_few<WEIGHTS, 32, 2>(p, r);
        else route_few<WEIGHTS, 8, 8>(p, r);
    } else if (E <= 256) {
        route_few<WEIGHTS, 32, 8>(p, r);
    } else {
        uint32_t* key = scratch + warp * E;
        for (int t = warp; t < p.T; t += WARPS) {
            for (int e = lane; e < E; e += 32) key[e] = order_key(logit(p, t, e));
            __syncwarp();
            int pick = -1;
            float val = 0.f, top = 0.f, all = 0.f;
            for (int j = 0; j < k; ++j) {
                uint32_t best = 0, m;
                int at = 0;
                for (int e = lane; e < E; e += 32)
                    if (key[e] > best) best = key[e], at = e;
                const int e = pick_of(best, at, m);
                if (e < 0) break;
                if (j == 0) {
                    top = key_value(m);
                    if (WEIGHTS && !p.renorm)
                        for (int i = lane; i < E; i += 32)
                            if (key[i] != 0) all += expf(key_value(key[i]) - top);
                }
                __syncwarp();
                if (e % 32 == lane) key[e] = 0;
                if (lane == j) pick = e, val = key_value(m);
                __syncwarp();
            }
            record<WEIGHTS>(p, r, t, pick, val, top, all);
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 0) {
        // the experts' first picks and groups: a lane has `each` neighbouring experts
        const int each = (E + 31) / 32, e0 = min(lane * each, E), e1 = min(e0 + each, E);
        const auto count = [&](int e) { return __popc(r.tokens[2 * e]) + __popc(r.tokens[2 * e + 1]); };
        int own = 0;  // picks in the upper half, groups in the lower (both below 2^15)
        for (int e = e0; e < e1; ++e) {
            const int c = count(e);
            own += c << 16 | (c + MAX_ROWS - 1) / MAX_ROWS;
        }
        int before = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += o;
        }
        if (lane == 31) *r.n_active = before & 0xffff, r.first[before & 0xffff] = before >> 16;
        before -= own;
        int a = before & 0xffff, at = before >> 16;
        for (int e = e0; e < e1; ++e) {
            const int c = count(e);
            r.base[e] = at;
            for (int i = 0; i < c; i += MAX_ROWS, ++a) r.active[a] = (uint16_t)e, r.first[a] = at + i;
            at += c;
        }
    }
    __syncthreads();
    // every pick's place: its token's rank among the expert's
    for (int i = threadIdx.x; i < picks; i += THREADS) {
        const int e = r.expert[i], t = i / k;
        if (e == NONE) continue;
        const unsigned lo = r.tokens[2 * e], hi = r.tokens[2 * e + 1], below = (1u << (t % 32)) - 1;
        r.pick[r.base[e] + (t < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below))] = (uint16_t)i;
    }
    __syncthreads();
}

// The tokens' sums of a slab of 64 columns: 8 columns of a token a thread.
template <bool BF16>
__device__ __forceinline__ void combine(const LayerParams& p, const Routes& r, int slab)
{
    for (int i = threadIdx.x; i < p.T * (SLAB / 8); i += 32 * MMA_WARPS) {
        const int t = i / (SLAB / 8), col = slab * SLAB + i % (SLAB / 8) * 8, n = min(8, p.D - col);
        if (n <= 0) continue;
        float v[8] = {}, res[8] = {};
        if (p.R) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < n)
                    res[c] = p.out_f32 ? static_cast<const float*>(p.R)[(int64_t)t * p.ldr + col + c]
                                       : from_16<BF16>(static_cast<const uint16_t*>(p.R)[(int64_t)t * p.ldr + col + c]);
        }
        // (four picks' rows under way at once; those of picks that are none are there and left out)
        for (int j0 = 0; j0 < p.k; j0 += 4) {
            float4 lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = t * p.k + min(j0 + i, p.k - 1);
                const float4* src = reinterpret_cast<const float4*>(p.y + (in_range(q, p.T * p.k) ? (int64_t)q * p.Dp : 0) + col);
                lo[i] = __ldcg(src), hi[i] = __ldcg(src + 1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = t * p.k + min(j0 + i, p.k - 1);
                if (j0 + i >= p.k || r.expert[q] == NONE) continue;
                const float w = r.weight[q];
                float y[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
                if (p.bias) {
                    const uint16_t* b = p.bias + (int64_t)r.expert[q] * p.D + col;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < n) y[c] += from_16<BF16>(b[c]);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] += w * y[c];
            }
        }
        if (p.R)
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] += res[c];
        if (p.out_f32) {
            float* o = static_cast<float*>(p.out) + (int64_t)t * p.ldo + col;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < n) o[c] = v[c];
        } else {
            uint16_t* o = static_cast<uint16_t*>(p.out) + (int64_t)t * p.ldo + col;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < n) o[c] = to_16<BF16>(v[c]);
        }
    }
}

// A stage's products for 16 columns and N tiles of 8 rows.
template <bool GATED, bool BF16, int N>
__device__ __forceinline__ void products(float (&acc)[MAX_TILES][2][4], uint32_t at_w, uint32_t at_x, int fg, int lane)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t wf[4][4], xf[N][2][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // matrices (k 0..7, f 0..7), (k 0..7, f 8..15), (k 8..15, f 0..7), (k 8..15, f 8..15)
            const int kr = h * (DEPTH / 2) + s * 16 + lane / 16 * 8 + lane % 8, c = lane / 8 % 2;
            if (GATED)
                ldsm_x4_trans(at_w + fg / 2 * (W_BYTES / 2) + kr * 64 + (((fg % 2 * 2 + c) ^ (kr / 2 & 3)) * 16), wf[s]);
            else
                ldsm_x4_trans(at_w + kr * 128 + (((fg * 2 + c) ^ (kr & 7)) * 16), wf[s]);
        }
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s)  // rows 8 t .. 8 t + 7, four chunks of 8 of k
                ldsm_x4(at_x + (t * 8 + lane % 8) * ROW_BYTES + (h * 8 + s * 4 + lane / 8) * 16, xf[t][s]);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < N; ++t)
                mma_16816<BF16>(acc[t][s & 1], wf[s], xf[t][s / 2][s % 2 * 2], xf[t][s / 2][s % 2 * 2 + 1]);
    }
}

// UP: H = act(X W1 + b1), else Y = H W2 and the tokens' sums.  Stage: [128 of the reduced
// dimension][64 columns] of W, swizzled by the TMA (128-byte rows; GATED, UP only: 32 columns of the gate,
// then 32 of the up half, each in 64-byte rows), and [row][128] of X or H.
template <bool UP, bool GATED, bool BF16>
__global__ void __launch_bounds__(THREADS, 2) layer_kernel(const __grid_constant__ CUtensorMap tmW, LayerParams p)
{
    constexpr int COLS = GATED ? SLAB / 2 : SLAB;  // output columns of an item
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring_w = smem_u32(smem), ring_x = ring_w + p.stages * W_BYTES;
    const int x_bytes = p.rows_cap * ROW_BYTES;
    float* const sums = reinterpret_cast<float*>(smem + p.stages * (W_BYTES + x_bytes));  // [rows_cap][PAD]
    const Routes r = carve(reinterpret_cast<uint8_t*>(sums + p.rows_cap * PAD), p.T * p.k, p.E);
    __shared__ uint64_t full_bar[MAX_STAGES], empty_bar[MAX_STAGES], never_bar;
    __shared__ int is_last;
    __shared__ volatile int abort_flag;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&full_bar[i]), 1 + 32);  // the weights' bytes, and each lane's copies of rows
            mbar_init(smem_u32(&empty_bar[i]), MMA_WARPS / 2);
        }
        mbar_init(smem_u32(&never_bar), 1);
        abort_flag = 0;
        mbar_fence_init();
        prefetch_tensormap(&tmW);
    }
    if (UP) {
        grid_dependency_wait();
        grid_dependents_launch();
    }
    // (the second kernel starts once every CTA of the first has got here: what came before that one,
    // the logits among it, is complete, and only H is not)
    route<!UP>(p, r, reinterpret_cast<uint32_t*>(smem));
    fence_proxy_async_shared();  // (the router's words lie where the TMA writes)
    __syncthreads();

    const int n_act = *r.n_active;
    const int K = UP ? p.D : p.F;
    const int steps = (K + DEPTH - 1) / DEPTH;
    const int items = n_act * p.slabs;
    const auto gave_up = [&](int code) {
        if (lane == 0) atomicCAS(p.status, 0, code);
        abort_flag = 1;
    };
    bool dead = false;

    if (warp == MMA_WARPS) {
        // ---------------------------------------------------------------- weights
        // (whole warps walk and one elected lane issues)
        int stage = 0;
        uint32_t phase = 0;
        for (int item = blockIdx.x; item < items && !dead; item += gridDim.x) {
            const int a = item / p.slabs, f = (item - a * p.slabs) * COLS, e = r.active[a];
            for (int step = 0; step < steps; ++step) {
                // (a full ring is emptied once the first kernel has ended: the wait's limit starts there)
                if (!UP && stage == 0 && phase == 1) grid_dependency_wait();
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty_bar[stage]), phase ^ 1, p.limit_ns, &abort_flag))) {
                    gave_up(kDevTimeoutProducer);
                    dead = true;
                    break;
                }
                if (elect_one()) {
                    const uint32_t bar = smem_u32(&full_bar[stage]), at = ring_w + stage * W_BYTES;
                    mbar_arrive_expect_tx(bar, W_BYTES);
                    tma_load_3d(at, &tmW, bar, f, step * DEPTH, e);
                    if (GATED) tma_load_3d(at + W_BYTES / 2, &tmW, bar, p.F + f, step * DEPTH, e);
                }
                __syncwarp();
                if (++stage == p.stages) stage = 0, phase ^= 1;
            }
        }
    } else if (warp == MMA_WARPS + 1) {
        // ---------------------------------------------------------------- rows
        if (!UP) {
            grid_dependency_wait();  // (the weights do not: they are under way before the first kernel has ended)
            grid_dependents_launch();
        }
        constexpr int LINE = DEPTH / 8;  // 16-byte chunks of a row: a lane has the same one of every second row
        const int c = lane % LINE, r0 = lane / LINE;
        const uint16_t* const rows = UP ? p.x : p.h;
        int stage = 0;
        uint32_t phase = 0;
        for (int item = blockIdx.x; item < items && !dead; item += gridDim.x) {
            const int a = item / p.slabs, first = r.first[a], n_rows = r.first[a + 1] - first;
            // lane i: where row i starts
            const int pick = r.pick[first + min(lane, n_rows - 1)];
            const int64_t starts = !in_range(pick, p.T * p.k) ? 0 : UP ? (int64_t)(pick / p.k) * p.ldx : (int64_t)pick * p.Fp;
            const auto source = [&](int row) { return rows + __shfl_sync(0xffffffffu, starts, row) + c * 8; };
            const uint16_t* src[4];  // of the first eight rows
#pragma unroll
            for (int i = 0; i < 4; ++i) src[i] = source(r0 + 2 * i);
            for (int step = 0; step < steps; ++step) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty_bar[stage]), phase ^ 1, p.limit_ns, &abort_flag))) {
                    gave_up(kDevTimeoutProducer);
                    dead = true;
                    break;
                }
                const int bytes = 2 * max(0, min(8, (UP ? K : p.Fp) - step * DEPTH - c * 8));  // of this chunk
                const uint32_t at = ring_x + stage * x_bytes + c * 16;
                // (what lies in a tile's rows behind the last stays: their products are not read)
                const auto copy = [&](int row, const uint16_t* from) {
                    if (row < n_rows) copy_async_16(at + row * ROW_BYTES, bytes > 0 ? from + step * DEPTH : rows, bytes);
                };
#pragma unroll
                for (int i = 0; i < 4; ++i) copy(r0 + 2 * i, src[i]);
#pragma unroll 4
                for (int i = 8; i < n_rows; i += 2) copy(i + r0, source(i + r0));
                copy_async_arrive(smem_u32(&full_bar[stage]));
                if (++stage == p.stages) stage = 0, phase ^= 1;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
    // -------------------------------------------------------------------- products
    if (!UP) grid_dependency_wait();  // (the limit of the waits below starts when the first kernel has ended)
    if (p.test_stall) {
        (void)mbar_wait(smem_u32(&never_bar), 0, p.limit_ns);
        gave_up(kDevTimeoutEpilogue);
        dead = true;
    }
    // a warp has 16 columns of every second stage: its latencies are another stage's time
    const int fg = warp % 4, kh = warp / 4;
    int stage = 0;
    uint32_t phase = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int a = item / p.slabs, slab = item - a * p.slabs;
        const int first = r.first[a], n_rows = r.first[a + 1] - first, tiles = (n_rows + 7) / 8;
        for (int step0 = 0; step0 < steps; step0 += RESTART) {
            float acc[MAX_TILES][2][4];  // even and odd steps of 16: an MMA takes 60 cycles to the next of its sum
#pragma unroll
            for (int t = 0; t < MAX_TILES; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[t][i / 4][i % 4] = 0.f;
            const int step1 = min(step0 + RESTART, steps);
            for (int step = step0; step < step1 && !dead; ++step) {
                if ((stage & 1) == kh) {
                    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full_bar[stage]), phase, p.limit_ns, &abort_flag))) {
                        gave_up(kDevTimeoutMma);
                        dead = true;
                        break;
                    }
                    const uint32_t at_w = ring_w + stage * W_BYTES, at_x = ring_x + stage * x_bytes;
                    switch (tiles) {
                    case 1: products<GATED, BF16, 1>(acc, at_w, at_x, fg, lane); break;
                    case 2: products<GATED, BF16, 2>(acc, at_w, at_x, fg, lane); break;
                    case 3: products<GATED, BF16, 3>(acc, at_w, at_x, fg, lane); break;
                    default: products<GATED, BF16, 4>(acc, at_w, at_x, fg, lane); break;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&empty_bar[stage]));
                }
                if (++stage == p.stages) stage = 0, phase ^= 1;
            }
#pragma unroll
            for (int t = 0; t < MAX_TILES; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][0][i] += acc[t][1][i];
            // the even and the odd stages, [row][column]; on top of the stretches before
            const int f = fg * 16 + lane / 4, row = lane % 4 * 2;
            if (kh == 1)
#pragma unroll
                for (int t = 0; t < MAX_TILES; ++t)
                    if (t < tiles) {
                        float* s = sums + (t * 8 + row) * PAD + f;
                        if (step0 == 0)
                            s[0] = acc[t][0][0], s[PAD] = acc[t][0][1], s[8] = acc[t][0][2], s[PAD + 8] = acc[t][0][3];
                        else
                            s[0] += acc[t][0][0], s[PAD] += acc[t][0][1], s[8] += acc[t][0][2], s[PAD + 8] += acc[t][0][3];
                    }
            named_barrier(1, 32 * MMA_WARPS);
            if (kh == 0)
#pragma unroll
                for (int t = 0; t < MAX_TILES; ++t)
                    if (t < tiles) {
                        float* s = sums + (t * 8 + row) * PAD + f;
                        s[0] += acc[t][0][0], s[PAD] += acc[t][0][1], s[8] += acc[t][0][2], s[PAD + 8] += acc[t][0][3];
                    }
            named_barrier(1, 32 * MMA_WARPS);
        }
        for (int q = threadIdx.x; q < n_rows * (COLS / 8) && !dead; q += 32 * MMA_WARPS) {
            const int i = q / (COLS / 8), c0 = q % (COLS / 8) * 8, pick = r.pick[first + i], col = slab * COLS + c0;
            if (!in_range(pick, p.T * p.k)) continue;
            const float* s = sums + i * PAD + c0;
            float v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = s[c];
            if constexpr (UP) {
                const int e = r.active[a];
                if (p.bias)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (col + c < p.F) v[c] += from_16<BF16>(p.bias[(int64_t)e * p.Fw + col + c]);
                if constexpr (GATED) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float up = s[SLAB / 2 + c];
                        if (p.bias && col + c < p.F) up += from_16<BF16>(p.bias[(int64_t)e * p.Fw + p.F + col + c]);
                        v[c] = silu(v[c]) * up;
                    }
                } else {
                    activate(v, p.act);
                }
                // (columns past F are zero, whatever W holds there: the gate's next ones are the up half's)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (col + c >= p.F) v[c] = 0.f;
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    w[c] = to_16<BF16>(v[2 * c]) | (uint32_t)to_16<BF16>(v[2 * c + 1]) << 16;
                if (in_range(col + 7, p.Fp))
                    *reinterpret_cast<uint4*>(p.h + (int64_t)pick * p.Fp + col) = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (in_range(col + 7, p.Dp)) {
                float4* o = reinterpret_cast<float4*>(p.y + (int64_t)pick * p.Dp + col);
                __stcg(o, make_float4(v[0], v[1], v[2], v[3]));
                __stcg(o + 1, make_float4(v[4], v[5], v[6], v[7]));
            }
        }
        if constexpr (UP) {
            named_barrier(1, 32 * MMA_WARPS);  // (the sums are read before the next item's are written)
        } else {
            // (one addition orders what every thread before the barrier has written)
            named_barrier(1, 32 * MMA_WARPS);
            if (threadIdx.x == 0) {
                const int last = add_acq_rel(p.counters + slab, 1u) == (unsigned)(n_act - 1);
                if (last) p.counters[slab] = 0;  // ready for the next launch
                is_last = last;
            }
            named_barrier(1, 32 * MMA_WARPS);
            if (is_last && !dead) combine<BF16>(p, r, slab);
        }
    }
    if constexpr (!UP) {
        if (n_act == 0 && !dead)  // no token goes anywhere
            for (int slab = blockIdx.x; slab < p.slabs; slab += gridDim.x) combine<BF16>(p, r, slab);
    }
    }
    if (__syncthreads_or(dead ? 1 : 0)) grace_period(2000000ull);  // (copies under way land before the exit)
}

// One matrix an expert, [E][K][N] with N contiguous: boxes of DEPTH rows of `box` columns.
bool encode_experts(CUtensorMap* map, const void* w, bool bf16, int64_t N, int64_t K, int64_t E, int64_t ld, int64_t stride,
                    int box)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)K, (cuuint64_t)E};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(E > 1 ? stride : ld) * 2};
    const cuuint32_t boxes[3] = {(cuuint32_t)box, DEPTH, 1}, estr[3] = {1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(w), dims,
               strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               box == SLAB ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool UP, bool GATED, bool BF16>
cudaError_t launch_typed(const CUtensorMap& map, const LayerParams& p, int grid, int smem, cudaStream_t s)
{
    auto kern = layer_kernel<UP, GATED, BF16>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, SMEM_ONE, allowed, true);
    return e != cudaSuccess ? e : launch_dependent(kern, dim3(grid), dim3(THREADS), smem, s, map, p);
}

int padded(int n) { return (n + SLAB - 1) / SLAB * SLAB; }

}  // namespace

size_t moe_layer_ws_bytes(const LayerArgs& a)
{
    return (size_t)a.T * a.k * (padded(a.F) * sizeof(uint16_t) + padded(a.D) * sizeof(float));
}

int launch_moe_layer(const LayerArgs& a, void* ws, unsigned* counters, int num_sms, int* dev_status, uint64_t limit_ns,
                     int test_stall, cudaStream_t s, int* launches)
{
    LayerParams p = {};
    p.T = a.T, p.E = a.E, p.k = a.k, p.D = a.D, p.F = a.F, p.Fw = a.Fw;
    p.logits = a.logits, p.ldl = a.ldl, p.logits_dtype = a.logits_dtype, p.renorm = a.renormalize;
    p.x = static_cast<const uint16_t*>(a.x), p.ldx = a.ldx;
    p.R = a.R, p.ldr = a.ldr;
    p.out = a.out, p.ldo = a.ldo;
    p.act = a.act, p.out_f32 = a.out_f32 ? 1 : 0;
    p.Fp = padded(a.F), p.Dp = padded(a.D);
    p.status = dev_status, p.limit_ns = limit_ns, p.test_stall = test_stall;
    const int picks = a.T * a.k;
    p.y = static_cast<float*>(ws);
    p.h = reinterpret_cast<uint16_t*>(p.y + (size_t)picks * p.Dp);
    p.counters = counters;
    p.rows_cap = a.T < MAX_ROWS ? (a.T + 7) / 8 * 8 : MAX_ROWS;
    // Bytes in flight decide: 128 KiB of weights an SM.  The second kernel has two CTAs of four stages an SM.
    // The first has one of six or eight, which leaves room for the first half of the second kernel's CTAs: they route
    // and fill their rings meanwhile.  With stages too large for that (more than 16 tokens): two CTAs of four
    // stages each, or one of as many as fit.
    const int stage = W_BYTES + p.rows_cap * ROW_BYTES, fixed = 1024 + p.rows_cap * PAD * 4 + routes_bytes(picks, a.E);
    const bool gated = a.act == GEMM_ACT_SWIGLU;
    const int most = most_groups(picks, a.E);
    const int up_slabs = p.Fp / (gated ? SLAB / 2 : SLAB), down_slabs = p.Dp / SLAB;
    int per_sm = 2, stages = (SMEM_TWO - fixed) / stage;
    if (stages < 4) per_sm = 1, stages = (SMEM_ONE - fixed) / stage;
    stages = stages > MAX_STAGES ? MAX_STAGES : stages / 2 * 2;
    if (per_sm == 2) stages = 4;
    if (stages < 2 || stages * stage < WARPS * a.E * 4) return GEMM_ERR_UNSUPPORTED;  // (the router's keys lie in the ring)
    int up_stages = stages, up_per_sm = per_sm;
    const int beside = (2 * SMEM_TWO - (stages * stage + fixed) - fixed) / stage / 2 * 2;
    if (per_sm == 2 && beside >= 6) up_stages = beside < MAX_STAGES ? beside : MAX_STAGES, up_per_sm = 1;
    const auto smem = [&](int n) { return n * stage + fixed; };
    const auto grid = [&](int slabs, int ctas) {
        const int64_t items = (int64_t)most * slabs, fit = ctas * num_sms;
        return (int)(items < fit ? items : fit);
    };
    CUtensorMap up, down;
    if (!encode_experts(&up, a.w1, a.bf16, a.Fw, a.D, a.E, a.ldw1, a.w1_stride, gated ? SLAB / 2 : SLAB) ||
        !encode_experts(&down, a.w2, a.bf16, a.D, a.F, a.E, a.ldw2, a.w2_stride, SLAB))
        return GEMM_ERR_CUDA;
    p.bias = static_cast<const uint16_t*>(a.b1);
    p.slabs = up_slabs, p.stages = up_stages;
    cudaError_t e = a.bf16 ? (gated ? launch_typed<true, true, true>(up, p, grid(p.slabs, up_per_sm), smem(p.stages), s)
                                    : launch_typed<true, false, true>(up, p, grid(p.slabs, up_per_sm), smem(p.stages), s))
                           : (gated ? launch_typed<true, true, false>(up, p, grid(p.slabs, up_per_sm), smem(p.stages), s)
                                    : launch_typed<true, false, false>(up, p, grid(p.slabs, up_per_sm), smem(p.stages), s));
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    p.bias = static_cast<const uint16_t*>(a.b2);
    p.slabs = down_slabs, p.stages = stages;
    e = a.bf16 ? launch_typed<false, false, true>(down, p, grid(p.slabs, per_sm), smem(p.stages), s)
               : launch_typed<false, false, false>(down, p, grid(p.slabs, per_sm), smem(p.stages), s);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

}  // namespace gemm_gb300
