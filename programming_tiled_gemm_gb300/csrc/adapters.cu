// The narrow half of a forward product with low-rank adapters: U[m] = s_i (X[m] A_i), i the row's
// adapter, rounded to 16 bits as an operand of the product that follows (linear_pair.h, linear_few.cu), and
// for that product's tiles the lists of their adapters and which of these have a B with infinities or NaN.
//
// A few rows or a short K (shrink_rows_kernel): a cluster a row, K shared by its CTAs, FMAs in fp32; bound by the
// reads of A, 16 bytes a thread.  More (shrink_groups_kernel): a cluster takes up to 64 rows of ONE adapter,
// wherever they lie, and shares K; so every A and every row of X is read once, whatever the rows' order.
// Which rows is found by every CTA for itself, by two passes over the rows' indices.  A ring of asynchronous
// copies brings them, 128 of K a stage, and mma.sync multiplies (rows of other adapters would only be masked
// on tcgen05's 128 or 256 rows, and the rank is narrower still).  The CTAs' parts of K are added in order
// through distributed shared memory.
//
// Measured (bf16, GPU time): 32 rows of 16 adapters, K 4096, rank 16: 4 us (2 MB of A: latency); 8192 rows in
// runs of one adapter, K 4096, rank 64: 30 us (71 MB, 2.4 TB/s: counting the rows 3.6, finding the group 3, the loop 16,
// the sums 3).  Dropped: tiles of 64 neighbouring rows with all their adapters (512 rows of 16 adapters at random, with
// the product: 94 us instead of 41); twice the CTAs a group for those rows (with the product 210 us instead of 200).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear.h"
#include "linear_math.h"
#include "ptx.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(adapters)

namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int MAX_CLUSTER = 8;

struct ShrinkParams {
    int M, K, Nw, n, r, rs;
    const uint16_t* X;
    int64_t ldx;
    const uint16_t* A;
    int64_t lda, a_stride;
    const uint16_t* B;
    int64_t ldb, b_stride;
    const int32_t* adapters;
    const float* scales;
    uint16_t* u;
    int* tiles;
    uint16_t* slot;
    uint8_t* bad;
    // clusters of U; after their CTAs come `lists` that make a list each, and those that look B through
    int tile_rows, cluster, work, lists;
};

__device__ __forceinline__ int adapter_of(const ShrinkParams& p, int m)
{
    const int id = m < p.M ? p.adapters[m] : -1;
    return id >= 0 && id < p.n ? id : -1;
}

// The list of one row tile, by one block: every adapter once, in the order of its first row.
__device__ __forceinline__ void make_list(const ShrinkParams& p, int tile)
{
    __shared__ __align__(16) int ids[THREADS];
    __shared__ int place[THREADS], before[WARPS];
    const int j = threadIdx.x, warp = j / 32, lane = j % 32, row = tile * p.tile_rows + j;
    const int id = j < p.tile_rows ? adapter_of(p, row) : -1;
    ids[j] = id;
    __syncthreads();
    int first = j;
#pragma unroll 8
    for (int i = 0; i < THREADS; i += 4) {
        const int4 o = *reinterpret_cast<const int4*>(&ids[i]);
        const int hit = o.x == id ? i : o.y == id ? i + 1 : o.z == id ? i + 2 : o.w == id ? i + 3 : j;
        first = min(first, hit);
    }
    const bool is = id >= 0 && first == j;
    const unsigned who = __ballot_sync(0xffffffffu, is);
    if (lane == 0) before[warp] = __popc(who);
    __syncthreads();
    int at = __popc(who & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += before[w];
        all += before[w];
    }
    place[j] = at;
    __syncthreads();
    int* list = p.tiles + (int64_t)tile * (1 + p.tile_rows);
    if (is) list[1 + at] = id;
    if (j == 0) list[0] = all;
    if (j < p.tile_rows && row < p.M && in_range(row, p.M)) p.slot[row] = id >= 0 ? (uint16_t)place[first] : (uint16_t)0xffff;
}

// Whether B holds infinities or NaN (exponents of ones): the used adapters' parts, shared by `ctas` CTAs.
// (It brings them into L2 for the product, too.)
template <bool BF16>
__device__ __forceinline__ void look_through(const ShrinkParams& p, int cta, int ctas)
{
    constexpr uint32_t EXP = BF16 ? 0x7f807f80u : 0x7c007c00u;
    constexpr int WORDS = kMaxAdapters / 32, FLY = 4;
    static_assert(WORDS == THREADS, "a word of the adapters' bits a thread");
    __shared__ unsigned used[WORDS];
    __shared__ int upto[WARPS];  // used adapters of the warps' words, summed
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    used[threadIdx.x] = 0;
    __syncthreads();
    for (int m = threadIdx.x; m < p.M; m += 8 * THREADS) {
        int id[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) id[i] = adapter_of(p, m + i * THREADS);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (id[i] >= 0 && (i == 0 || id[i] != id[i - 1])) atomicOr(&used[id[i] / 32], 1u << (id[i] % 32));
    }
    __syncthreads();
    const int own = __popc(used[threadIdx.x]);
    int before = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) upto[warp] = before;
    __syncthreads();
    int all = 0;
    before -= own;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += upto[w];
        all += upto[w];
    }
    __shared__ int who;
    // parts of an adapter's B, a task each: about as many tasks as CTAs, or more where B is long.  (32 whatever their
    // number: 32 x 4096 x 4096 with 16 adapters of rank 16, residual, 25.4 us instead of 24.4.)
    int parts = 1;
    while (parts < kAdapterParts && (parts * all < ctas || (int64_t)p.r * (p.Nw / 8) / parts > 1 << 16)) parts *= 2;
    for (int task = cta; task < all * parts; task += ctas) {
        // the task's adapter: the thread whose word holds it
        const int nth = task / parts, part = task % parts;
        if (nth >= before && nth < before + own) {
            unsigned bits = used[threadIdx.x];
            for (int i = before; i < nth; ++i) bits &= bits - 1;
            who = threadIdx.x * 32 + __ffs(bits) - 1;
        }
        __syncthreads();
        const int id = who, all_chunks = p.Nw / 8 + (p.Nw % 8 != 0);
        const int q0 = (int)((int64_t)all_chunks * part / parts), chunks = (int)((int64_t)all_chunks * (part + 1) / parts) - q0;
        int hit = 0;
        for (int q = threadIdx.x; q < p.r * chunks; q += FLY * THREADS) {
            uint4 v[FLY];
#pragma unroll
            for (int i = 0; i < FLY; ++i) {
                const int at = q + i * THREADS, k = at / max(chunks, 1), c = (q0 + at - k * chunks) * 8;
                v[i] = make_uint4(0, 0, 0, 0);
                if (at >= p.r * chunks || !in_range(c, p.Nw)) continue;
                const uint16_t* b = p.B + id * p.b_stride + (int64_t)k * p.ldb + c;
                if (c + 8 <= p.Nw) {
                    v[i] = __ldg(reinterpret_cast<const uint4*>(b));
                } else {
                    for (int j = 0; c + j < p.Nw; ++j) hit |= (b[j] & EXP & 0xffffu) == (EXP & 0xffffu);
                }
            }
#pragma unroll
            for (int i = 0; i < FLY; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t e = w[j] & EXP;
                    hit |= (e & 0xffffu) == (EXP & 0xffffu) || (e >> 16) == (EXP >> 16);
                }
            }
        }
        hit = __syncthreads_or(hit);
        const int flags = kAdapterParts / parts;
        if ((int)threadIdx.x < flags) p.bad[(int64_t)id * kAdapterParts + part * flags + threadIdx.x] = (uint8_t)(hit != 0);
    }
}

template <bool BF16>
__device__ __forceinline__ float2 two(uint32_t u)
{
    if (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}

// ------------------------------------------------------------------ a cluster a row

template <bool BF16>
__global__ void __launch_bounds__(THREADS) shrink_rows_kernel(ShrinkParams p)
{
    __shared__ float red[WARPS][kMaxAdapterRank];
    __shared__ float part[MAX_CLUSTER][kMaxAdapterRank];  // the CTAs' sums, in the first one's
    grid_dependency_wait();
    grid_dependents_launch();
    const int C = p.cluster, rank = blockIdx.x % C, m = blockIdx.x / C;
    if (m >= p.work) {
        const int extra = blockIdx.x - p.work * C;
        if (extra < p.lists) make_list(p, extra);
        else if (p.bad) look_through<BF16>(p, extra - p.lists, gridDim.x - p.work * C - p.lists);
        return;
    }
    const int id = adapter_of(p, m);
    if (id < 0) return;  // (the whole cluster)
    if (C > 1) cluster_arrive();  // (the first CTA is there before the others write to it)
    const float scale = p.scales ? p.scales[id] : 1.f;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // a lane has eight ranks of every `per`-th row of A
    const int chunks = p.r / 8;
    int pitch = 1;
    while (pitch < chunks) pitch *= 2;
    const int c = lane % pitch, per = 32 / pitch * WARPS;
    const int k0 = (int)((int64_t)p.K * rank / C), k1 = (int)((int64_t)p.K * (rank + 1) / C);
    const uint16_t* x = p.X + (int64_t)m * p.ldx;
    const uint16_t* A = p.A + id * p.a_stride + c * 8;
    float acc[8] = {};
    if (c < chunks) {
        constexpr int FLY = 8;
        for (int k = k0 + warp * (32 / pitch) + lane / pitch; k < k1; k += FLY * per) {
            uint4 v[FLY];
            uint16_t xv[FLY];
#pragma unroll
            for (int i = 0; i < FLY; ++i)
                if (k + i * per < k1) {
                    v[i] = __ldg(reinterpret_cast<const uint4*>(A + (int64_t)(k + i * per) * p.lda));
                    xv[i] = x[k + i * per];
                }
#pragma unroll
            for (int i = 0; i < FLY; ++i)
                if (k + i * per < k1) {
                    const float f = from_16<BF16>(xv[i]);
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 t = two<BF16>(w[q]);
                        acc[2 * q] = fmaf(f, t.x, acc[2 * q]);
                        acc[2 * q + 1] = fmaf(f, t.y, acc[2 * q + 1]);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        for (int d = pitch; d < 32; d *= 2) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
    if (lane < chunks)
#pragma unroll
        for (int i = 0; i < 8; ++i) red[warp][lane * 8 + i] = acc[i];
    __syncthreads();
    if (C > 1) cluster_wait();
    if ((int)threadIdx.x < p.r) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += red[w][threadIdx.x];
        const uint32_t at = smem_u32(&part[rank][threadIdx.x]);
        if (C > 1) st_shared_cluster_f32(mapa_shared(at, 0), s);
        else part[0][threadIdx.x] = s;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    if (rank != 0 || (int)threadIdx.x >= p.rs) return;
    float s = 0.f;
    if ((int)threadIdx.x < p.r) {
#pragma unroll
        for (int q = 0; q < MAX_CLUSTER; ++q)
            if (q < C) s += part[q][threadIdx.x];
        s *= scale;
    }
    if (in_range(m, p.M)) p.u[(int64_t)m * p.rs + threadIdx.x] = to_16<BF16>(s);
}

// ------------------------------------------------------------------ a cluster up to 64 rows of an adapter

constexpr int ROWS = 64;
constexpr int RING = 3;                    // stages
constexpr int depth_of(int rs) { return rs <= 64 ? 128 : 64; }  // of K a stage
constexpr int x_pitch(int rs) { return depth_of(rs) * 2 + 16; }  // bytes of a row of X: rows 16 bytes apart in the banks
constexpr int a_pitch(int rs) { return rs * 2 + 16; }
constexpr int group_stage(int rs) { return ROWS * x_pitch(rs) + depth_of(rs) * a_pitch(rs); }
constexpr int sums_bytes(int rs) { return (ROWS + WARPS * 16) * (rs + 1) * 4; }  // in the ring's place afterwards
constexpr int groups_smem(int rs) { return RING * group_stage(rs) > sums_bytes(rs) ? RING * group_stage(rs) : sums_bytes(rs); }

// The sum over the block's threads before this one, and of all.
__device__ __forceinline__ int sum_before(int v, int* per_warp, int& all)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    if (lane == 31) per_warp[warp] = s;
    __syncthreads();
    all = 0;
    s -= v;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) s += per_warp[w];
        all += per_warp[w];
    }
    __syncthreads();
    return s;
}

// The adapters of rows m .. m + 3 (m a multiple of 4), -1 past the last row.
__device__ __forceinline__ int4 four_adapters(const ShrinkParams& p, int m)
{
    if (m + 4 > p.M || (reinterpret_cast<uintptr_t>(p.adapters) & 15) != 0)
        return make_int4(adapter_of(p, m), adapter_of(p, m + 1), adapter_of(p, m + 2), adapter_of(p, m + 3));
    int4 v = *reinterpret_cast<const int4*>(p.adapters + m);
    v.x = v.x >= 0 && v.x < p.n ? v.x : -1, v.y = v.y >= 0 && v.y < p.n ? v.y : -1;
    v.z = v.z >= 0 && v.z < p.n ? v.z : -1, v.w = v.w >= 0 && v.w < p.n ? v.w : -1;
    return v;
}

// How many rows every adapter has: a word each in `counts`.
__device__ __forceinline__ void count_rows(const ShrinkParams& p, int* counts)
{
    constexpr int FLY = 4;
    for (int i = threadIdx.x; i < p.n; i += THREADS) counts[i] = 0;
    __syncthreads();
    for (int b = 0; b < p.M; b += FLY * 4 * THREADS) {
        int4 v[FLY];
#pragma unroll
        for (int i = 0; i < FLY; ++i) v[i] = four_adapters(p, b + (i * THREADS + (int)threadIdx.x) * 4);
#pragma unroll
        for (int i = 0; i < FLY; ++i) {
            // (a warp's 128 rows often have one adapter: one addition for all of them)
            const int first = __shfl_sync(0xffffffffu, v[i].x, 0);
            if (__all_sync(0xffffffffu, v[i].x == first && v[i].y == first && v[i].z == first && v[i].w == first)) {
                if (first >= 0 && threadIdx.x % 32 == 0) atomicAdd(&counts[first], 128);
                continue;
            }
            if (v[i].x >= 0) atomicAdd(&counts[v[i].x], 1);
            if (v[i].y >= 0) atomicAdd(&counts[v[i].y], 1);
            if (v[i].z >= 0) atomicAdd(&counts[v[i].z], 1);
            if (v[i].w >= 0) atomicAdd(&counts[v[i].w], 1);
        }
    }
    __syncthreads();
}

// The `group`-th of the adapters' groups of 64 rows: its adapter (-1: there are not as many), its rows in
// `rows` and their number.
__device__ __forceinline__ int find_group(const ShrinkParams& p, int group, const int* counts, int* rows, int& n_rows)
{
    __shared__ int per_warp[WARPS], found_id, found_chunk;
    constexpr int FLY = 4;
    if (threadIdx.x == 0) found_id = -1, found_chunk = 0;
    __syncthreads();
    // the adapter that holds the group: a thread has `each` neighbouring adapters
    const int each = (p.n + THREADS - 1) / THREADS, i0 = min((int)threadIdx.x * each, p.n), i1 = min(i0 + each, p.n);
    int own = 0, all;
    for (int i = i0; i < i1; ++i) own += (counts[i] + ROWS - 1) / ROWS;
    int before = sum_before(own, per_warp, all);
    if (group >= before && group < before + own)
        for (int i = i0; i < i1; ++i) {
            const int g = (counts[i] + ROWS - 1) / ROWS;
            if (group < before + g) {
                found_id = i, found_chunk = group - before;
                break;
            }
            before += g;
        }
    __syncthreads();
    const int id = found_id;
    if (id < 0) return -1;
    // its rows, in order: a warp has a stretch of them, 128 at a time
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int skip = found_chunk * ROWS, stretch = (p.M + 128 * WARPS - 1) / (128 * WARPS) * 128, m0 = warp * stretch;
    const int m1 = min(m0 + stretch, p.M);
    int mine = 0;
    for (int m = m0; m < m1; m += 128 * FLY) {
        int4 v[FLY];
#pragma unroll
        for (int i = 0; i < FLY; ++i)
            v[i] = m + 128 * i < m1 ? four_adapters(p, m + 128 * i + lane * 4) : make_int4(-1, -1, -1, -1);
#pragma unroll
        for (int i = 0; i < FLY; ++i) mine += (v[i].x == id) + (v[i].y == id) + (v[i].z == id) + (v[i].w == id);
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) per_warp[warp] = mine;
    __syncthreads();
    int at = -skip;
    all = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += per_warp[w];
        all += per_warp[w];
    }
    if (at + mine > 0)
        for (int m = m0; m < m1 && at < ROWS; m += 128) {
            const int4 v = four_adapters(p, m + lane * 4);
            const bool is[4] = {v.x == id, v.y == id, v.z == id, v.w == id};
            int place = at;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned who = __ballot_sync(0xffffffffu, is[j]);
                place += __popc(who & ((1u << lane) - 1));
                at += __popc(who);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (is[j]) {
                    if (place >= 0 && place < ROWS) rows[place] = m + lane * 4 + j;
                    ++place;
                }
        }
    n_rows = min(ROWS, all - skip);
    __syncthreads();
    return id;
}

// Warps: 16 of the rows x a part of every stage's K, more parts where there are fewer rows.
template <bool BF16, int RS>
__global__ void __launch_bounds__(THREADS, RS <= 64 ? 2 : 1) shrink_groups_kernel(ShrinkParams p)
{
    constexpr int NT = RS / 8, PITCH = a_pitch(RS), DEPTH = depth_of(RS), X_PITCH = x_pitch(RS), LINE = DEPTH / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int rows[ROWS];
    int* const counts = reinterpret_cast<int*>(smem + groups_smem(RS));
    grid_dependency_wait();
    grid_dependents_launch();
    const int C = p.cluster, rank = blockIdx.x % C;
    if (blockIdx.x / C >= p.work) {
        const int extra = blockIdx.x - p.work * C;
        if (extra < p.lists) make_list(p, extra);
        else if (p.bad) look_through<BF16>(p, extra - p.lists, gridDim.x - p.work * C - p.lists);
        return;
    }
    count_rows(p, counts);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int group = blockIdx.x / C;; group += p.work) {
        int n_rows = 0;
        const int id = find_group(p, group, counts, rows, n_rows);
        if (id < 0) return;  // (the whole cluster)
        const float scale = p.scales ? p.scales[id] : 1.f;
        const uint32_t ring = smem_u32(smem);
        const int kb = (p.K + DEPTH - 1) / DEPTH, kb0 = kb * rank / C, steps = kb * (rank + 1) / C - kb0;
        // 16 rows a warp, and `parts` warps share a stage's K
        const int tiles = n_rows <= 16 ? 1 : n_rows <= 32 ? 2 : 4, parts = WARPS / tiles, rg = warp % tiles, part = warp / tiles;
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
        // what a thread copies of every stage: the same 16 bytes of some rows of X and of some rows of A
        constexpr int XS = ROWS * LINE / THREADS, AS = DEPTH * NT / THREADS > 0 ? DEPTH * NT / THREADS : 1;
        const int xc = threadIdx.x % LINE, xr = threadIdx.x / LINE, ac = threadIdx.x % NT, ar = threadIdx.x / NT;
        const uint16_t* xp[XS];
#pragma unroll
        for (int i = 0; i < XS; ++i) {
            const int row = xr + i * (THREADS / LINE);
            xp[i] = p.X + (row < n_rows && in_range(rows[row], p.M) ? (int64_t)rows[row] * p.ldx : 0) + (int64_t)kb0 * DEPTH + xc * 8;
        }
        const uint16_t* ap = p.A + id * p.a_stride + (int64_t)(kb0 * DEPTH + ar) * p.lda + ac * 8;
        int l_step = 0;
        const auto load = [&] {
            if (l_step < steps) {
                const int k0 = (kb0 + l_step) * DEPTH;
                const uint32_t at = ring + l_step % RING * group_stage(RS);
                const int nx = 2 * max(0, min(8, p.K - k0 - xc * 8));
#pragma unroll
                for (int i = 0; i < XS; ++i) {
                    const int row = xr + i * (THREADS / LINE), n = row < n_rows ? nx : 0;
                    if (row < tiles * 16) copy_async_16(at + row * X_PITCH + xc * 16, n > 0 ? xp[i] + l_step * DEPTH : p.X, n);
                }
#pragma unroll
                for (int i = 0; i < AS; ++i) {
                    const int k = ar + i * (THREADS / NT);
                    if (DEPTH * NT < THREADS && k >= DEPTH) break;
                    const int n = k0 + k < p.K && ac * 8 < p.r && in_range(k0 + k, p.K) ? 16 : 0;
                    copy_async_16(at + ROWS * X_PITCH + k * PITCH + ac * 16,
                                  n > 0 ? ap + (int64_t)(l_step * DEPTH + i * (THREADS / NT)) * p.lda : p.A, n);
                }
                ++l_step;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = 0; i < RING - 1; ++i) load();
        for (int s = 0; s < steps; ++s) {
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
            __syncthreads();
            load();  // into the stage that was multiplied before the barrier
            const uint32_t xs = ring + s % RING * group_stage(RS), as = xs + ROWS * X_PITCH;
#pragma unroll 4
            for (int k = part * 16; k < DEPTH; k += parts * 16) {
                uint32_t xf[4];  // (rows 0..7, k 0..7), (8..15, 0..7), (0..7, 8..15), (8..15, 8..15)
                ldsm_x4(xs + (rg * 16 + lane % 16) * X_PITCH + (k + lane / 16 * 8) * 2, xf);
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t af[4];  // (k 0..7, ranks 0..7), (k 8..15, 0..7), (k 0..7, 8..15), (k 8..15, 8..15)
                    ldsm_x4_trans(as + (k + lane % 16) * PITCH + (t * 8 + lane / 16 * 8) * 2, af);
                    mma_16816<BF16>(acc[t], xf, af[0], af[1]);
                    mma_16816<BF16>(acc[t + 1], xf, af[2], af[3]);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // [row][rank] of the warps, of a stage's parts, then of the cluster's CTAs, in order
        constexpr int FP = RS + 1;
        float* const own = reinterpret_cast<float*>(smem) + ROWS * FP + warp * 16 * FP;
        float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) own[(lane / 4 + i / 2 * 8) * FP + t * 8 + lane % 4 * 2 + i % 2] = acc[t][i];
        __syncthreads();
        for (int q = threadIdx.x; q < n_rows * RS; q += THREADS) {
            const int i = q / RS, c = q % RS;
            const float* from = sums + ROWS * FP + i * FP + c;  // (row i: row i % 16 of warp i / 16)
            float v = 0.f;
            for (int h = 0; h < parts; ++h) v += from[h * tiles * 16 * FP];
            sums[i * FP + c] = v;
        }
        __syncthreads();
        if (C > 1) cluster_sync_all();
        for (int q = rank * THREADS + threadIdx.x; q < n_rows * RS; q += C * THREADS) {
            const int i = q / RS, c = q % RS;
            const uint32_t at = smem_u32(sums + i * FP + c);
            float t[MAX_CLUSTER], v = 0.f;
#pragma unroll
            for (int w = 0; w < MAX_CLUSTER; ++w)
                if (w < C) t[w] = C > 1 ? ld_shared_cluster_f32(mapa_shared(at, w)) : sums[i * FP + c];
#pragma unroll
            for (int w = 0; w < MAX_CLUSTER; ++w)
                if (w < C) v += t[w];
            if (in_range(rows[i], p.M)) p.u[(int64_t)rows[i] * RS + c] = to_16<BF16>(c < p.r ? v * scale : 0.f);
        }
        // (nobody leaves or writes over its sums while they are read)
        if (C > 1) cluster_sync_all();
        else __syncthreads();
    }
}

// `most`: of shared memory, that any launch of the kernel takes.
template <typename Kernel>
cudaError_t launch(Kernel kern, int smem, int most, std::atomic<uint64_t>* allowed, const ShrinkParams& p, int clusters,
                   cudaStream_t s)
{
    if (allowed) {
        const cudaError_t e = allow_smem(kern, most, *allowed);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * p.cluster), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool BF16, int RS>
cudaError_t launch_groups(const ShrinkParams& p, int clusters, cudaStream_t s)
{
    static std::atomic<uint64_t> allowed{0};
    // (behind the ring a word an adapter; as much as any number of them takes is asked for)
    static_assert(groups_smem(RS) + kMaxAdapters * 4 <= 232448 - 4096, "shared memory of a CTA");
    return launch(shrink_groups_kernel<BF16, RS>, groups_smem(RS) + p.n * 4, groups_smem(RS) + kMaxAdapters * 4, &allowed, p,
                  clusters, s);
}

}  // namespace

int launch_shrink(const LinArgs& a, const LinAdapt& ad, int num_sms, cudaStream_t stream, int* launches)
{
    ShrinkParams p = {};
    p.M = (int)a.M, p.K = (int)a.K, p.Nw = (int)a.Nw, p.n = ad.n, p.r = ad.r, p.rs = ad.rs;
    p.X = static_cast<const uint16_t*>(a.X), p.ldx = a.ldx;
    p.A = static_cast<const uint16_t*>(ad.A), p.lda = ad.lda, p.a_stride = ad.a_stride;
    p.B = static_cast<const uint16_t*>(ad.B), p.ldb = ad.ldb, p.b_stride = ad.b_stride;
    p.adapters = ad.adapters, p.scales = ad.scales;
    p.u = ad.u, p.tile_rows = ad.tile_rows;
    if (ad.tile_rows > 0) p.tiles = ad.tiles, p.slot = ad.slot, p.bad = ad.bad;
    p.lists = ad.tile_rows > 0 ? (p.M + ad.tile_rows - 1) / ad.tile_rows : 0;
    // A cluster a row reads its A for itself, rows of one adapter again from L2, but is done sooner than the
    // rows of an adapter are found.  us of the whole call with a cluster a row and with groups (adapters at
    // random; M x K x rank): 32 x 4096 x 16 24.5 25.5, 77 x 1000 x 24 15.8 20.0, 256 x 1024 x 16 19.8 19.5,
    // 64 x 4096 x 16 30.3 29.0, 256 x 4096 x 16 35.6 32.3, 32 x 4096 x 64 39.4 39.3, 128 x 4096 x 64 52.9 46.8
    const bool rows = a.M * a.K * ad.r <= (int64_t)4 << 20 || ad.tile_rows == 0;
    const int64_t groups = (a.M < ad.n ? a.M : ad.n) + a.M / ROWS, fit = (rows ? 4 : 2) * num_sms;  // at most, and CTAs
    p.work = rows ? p.M : (int)(groups < fit ? groups : fit);
    // K is shared by as many CTAs as fit at once and have some 256 (128) of it
    p.cluster = 1;
    while (p.cluster < MAX_CLUSTER && 2 * p.cluster * p.work <= fit && 2 * p.cluster * (rows ? 256 : 128) <= p.K) p.cluster *= 2;
    // (B is looked through beside the rest, by a CTA an SM)
    const int clusters = p.work + (p.lists > 0 ? (p.lists + num_sms + p.cluster - 1) / p.cluster : 0);
    cudaError_t e;
    if (rows) {
        e = a.bf16 ? launch(shrink_rows_kernel<true>, 0, 0, nullptr, p, clusters, stream)
                   : launch(shrink_rows_kernel<false>, 0, 0, nullptr, p, clusters, stream);
    } else {
        const auto groups_of = a.bf16 ? (p.rs == 16   ? launch_groups<true, 16>
                                         : p.rs == 32 ? launch_groups<true, 32>
                                         : p.rs == 64 ? launch_groups<true, 64>
                                                      : launch_groups<true, 128>)
                                      : (p.rs == 16   ? launch_groups<false, 16>
                                         : p.rs == 32 ? launch_groups<false, 32>
                                         : p.rs == 64 ? launch_groups<false, 64>
                                                      : launch_groups<false, 128>);
        e = groups_of(p, clusters, stream);
    }
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

}  // namespace gemm_gb300
