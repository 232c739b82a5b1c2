// The narrow half of a forward product with low-rank adapters: U[m] = s_i (X[m] A_i), i the row's
// adapter, rounded to 16 bits as an operand of the product that follows (linear_pair.h, linear_few.cu), and
// for that product's tiles the lists of their adapters and which of these have a B with infinities or NaN.
//
// Few rows (shrink_rows_kernel): a cluster a row, K shared by its CTAs, FMAs in fp32; bound by the reads of
// A, 16 bytes a thread.  Many rows (shrink_tiles_kernel): a cluster takes 64 rows and shares K; a ring of
// asynchronous copies brings 64 of K of X and of an adapter's A, for one adapter of the tile's rows after the
// other, and mma.sync multiplies them (the rank is too narrow a side for tcgen05's 128 or 256); a row takes the
// sums of its own adapter only, so that no adapter's NaN reaches another's rows.  Bound by X's bytes where
// requests lie together.  The CTAs' parts of K are added in order through distributed shared memory.
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
    for (int task = cta; task < all * kAdapterParts; task += ctas) {
        // the task's adapter: the thread whose word holds it
        const int nth = task / kAdapterParts, part = task % kAdapterParts;
        if (nth >= before && nth < before + own) {
            unsigned bits = used[threadIdx.x];
            for (int i = before; i < nth; ++i) bits &= bits - 1;
            who = threadIdx.x * 32 + __ffs(bits) - 1;
        }
        __syncthreads();
        const int id = who, q0 = (p.Nw + 7) / 8 * part / kAdapterParts, chunks = (p.Nw + 7) / 8 * (part + 1) / kAdapterParts - q0;
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
        if (threadIdx.x == 0) p.bad[(int64_t)id * kAdapterParts + part] = (uint8_t)(hit != 0);
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
    __shared__ float part[kMaxAdapterRank];
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
    if ((int)threadIdx.x < p.r) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += red[w][threadIdx.x];
        part[threadIdx.x] = s;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    if (rank == 0 && (int)threadIdx.x < p.rs) {
        float s = 0.f;
        if ((int)threadIdx.x < p.r) {
            const uint32_t at = smem_u32(&part[threadIdx.x]);
            float t[MAX_CLUSTER];
#pragma unroll
            for (int q = 0; q < MAX_CLUSTER; ++q)
                if (q < C) t[q] = C > 1 ? ld_shared_cluster_f32(mapa_shared(at, q)) : part[threadIdx.x];
#pragma unroll
            for (int q = 0; q < MAX_CLUSTER; ++q)
                if (q < C) s += t[q];
            if (p.scales) s *= p.scales[id];
        }
        if (in_range(m, p.M)) p.u[(int64_t)m * p.rs + threadIdx.x] = to_16<BF16>(s);
    }
    if (C > 1) cluster_sync_all();  // (nobody leaves while its sums are read)
}

// ------------------------------------------------------------------ a cluster 64 rows

constexpr int ROWS = 64;
constexpr int RING = 3;                    // stages
constexpr int depth_of(int rs) { return rs <= 64 ? 128 : 64; }  // of K a stage
constexpr int x_pitch(int rs) { return depth_of(rs) * 2 + 16; }  // bytes of a row of X: rows 16 bytes apart in the banks
constexpr int a_pitch(int rs) { return rs * 2 + 16; }
constexpr int tile_stage(int rs) { return ROWS * x_pitch(rs) + depth_of(rs) * a_pitch(rs); }
constexpr int tiles_smem(int rs) { return RING * tile_stage(rs); }
static_assert(tiles_smem(16) >= ROWS * (16 + 1) * 4 && tiles_smem(128) >= ROWS * (128 + 1) * 4, "the sums lie in the ring");

__device__ __forceinline__ void ldsm_x4(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Warps: 16 rows (of 64) x half of every stage's K.
template <bool BF16, int RS>
__global__ void __launch_bounds__(THREADS) shrink_tiles_kernel(ShrinkParams p)
{
    constexpr int NT = RS / 8, PITCH = a_pitch(RS), DEPTH = depth_of(RS), X_PITCH = x_pitch(RS), LINE = DEPTH / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) int ids[ROWS];
    __shared__ int list[ROWS], count;
    grid_dependency_wait();
    grid_dependents_launch();
    const int C = p.cluster, rank = blockIdx.x % C, tile = blockIdx.x / C;
    if (tile >= p.work) {
        const int extra = blockIdx.x - p.work * C;
        if (extra < p.lists) make_list(p, extra);
        else if (p.bad) look_through<BF16>(p, extra - p.lists, gridDim.x - p.work * C - p.lists);
        return;
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row0 = tile * ROWS;
    if ((int)threadIdx.x < ROWS) ids[threadIdx.x] = adapter_of(p, row0 + threadIdx.x);
    __syncthreads();
    if (warp == 0) {
        // the tile's adapters, in the order of their first rows
        int n = 0;
        for (int h = 0; h < ROWS; h += 32) {
            const int j = h + lane, id = ids[j];
            bool is = id >= 0;
            for (int i = 0; i < j; ++i) is = is && ids[i] != id;
            const unsigned who = __ballot_sync(0xffffffffu, is);
            if (is) list[n + __popc(who & ((1u << lane) - 1))] = id;
            n += __popc(who);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int adapters = count;
    if (adapters == 0) return;  // (the whole cluster)
    const uint32_t ring = smem_u32(smem);
    const int kb = (p.K + DEPTH - 1) / DEPTH, kb0 = kb * rank / C, nb = kb * (rank + 1) / C - kb0, steps = adapters * nb;
    const int rg = warp % 4, kh = warp / 4;
    const int id0 = ids[rg * 16 + lane / 4], id1 = ids[rg * 16 + lane / 4 + 8];  // of this thread's two rows
    float sum[NT][4], acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[t][i] = 0.f;
    // the loader's adapter and k-block, RING - 1 stages ahead
    int l_step = 0, l_adapter = 0, l_block = 0;
    const auto load = [&] {
        if (l_step < steps) {
            const int k0 = (kb0 + l_block) * DEPTH;
            const uint32_t at = ring + l_step % RING * tile_stage(RS);
#pragma unroll
            for (int i = 0; i < ROWS * LINE / THREADS; ++i) {
                const int q = threadIdx.x + i * THREADS, row = q / LINE, k = k0 + q % LINE * 8;
                int n = row0 + row < p.M ? max(0, min(8, p.K - k)) : 0;
                if (n > 0 && !in_range(row0 + row, p.M)) n = 0;
                copy_async_16(at + row * X_PITCH + q % LINE * 16, n > 0 ? p.X + (int64_t)(row0 + row) * p.ldx + k : p.X, 2 * n);
            }
            const uint16_t* A = p.A + list[l_adapter] * p.a_stride;
#pragma unroll
            for (int q = threadIdx.x; q < DEPTH * NT; q += THREADS) {
                const int k = q / NT, c = q % NT;
                int n = k0 + k < p.K && c * 8 < p.r ? 8 : 0;
                if (n > 0 && !in_range(k0 + k, p.K)) n = 0;
                copy_async_16(at + ROWS * X_PITCH + k * PITCH + c * 16, n > 0 ? A + (int64_t)(k0 + k) * p.lda + c * 8 : p.A, 2 * n);
            }
            ++l_step;
            if (++l_block == nb) l_block = 0, ++l_adapter;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < RING - 1; ++i) load();
    for (int d = 0, s = 0; d < adapters && nb > 0; ++d) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
        for (int b = 0; b < nb; ++b, ++s) {
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
            __syncthreads();
            load();  // into the stage that was multiplied before the barrier
            const uint32_t xs = ring + s % RING * tile_stage(RS), as = xs + ROWS * X_PITCH;
#pragma unroll
            for (int h = 0; h < DEPTH / 32; ++h) {
                const int k = kh * (DEPTH / 2) + h * 16;
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
        const int id = list[d];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (id0 == id) sum[t][0] = acc[t][0], sum[t][1] = acc[t][1];
            if (id1 == id) sum[t][2] = acc[t][2], sum[t][3] = acc[t][3];
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // [row][rank] of both halves, then of the cluster's CTAs, in order
    float* part = reinterpret_cast<float*>(smem);
    const int row = rg * 16 + lane / 4, col = lane % 4 * 2;
    constexpr int FP = RS + 1;
    for (int h = 0; h < 2; ++h) {
        if (kh == h)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float* o = part + (row + i / 2 * 8) * FP + t * 8 + col + i % 2;
                    *o = h ? *o + sum[t][i] : sum[t][i];
                }
        __syncthreads();
    }
    if (C > 1) cluster_sync_all();
    for (int q = rank * THREADS + threadIdx.x; q < ROWS * RS; q += C * THREADS) {
        const int i = q / RS, c = q % RS, id = ids[i];
        if (id < 0) continue;
        const uint32_t at = smem_u32(part + i * FP + c);
        float t[MAX_CLUSTER], v = 0.f;
#pragma unroll
        for (int w = 0; w < MAX_CLUSTER; ++w)
            if (w < C) t[w] = C > 1 ? ld_shared_cluster_f32(mapa_shared(at, w)) : part[i * FP + c];
#pragma unroll
        for (int w = 0; w < MAX_CLUSTER; ++w)
            if (w < C) v += t[w];
        if (p.scales) v *= p.scales[id];
        if (in_range(row0 + i, p.M)) p.u[(int64_t)(row0 + i) * RS + c] = to_16<BF16>(c < p.r ? v : 0.f);
    }
    if (C > 1) cluster_sync_all();  // (nobody leaves while its sums are read)
}

template <typename Kernel>
cudaError_t launch(Kernel kern, int smem, std::atomic<uint64_t>* allowed, const ShrinkParams& p, int clusters, cudaStream_t s)
{
    if (allowed) {
        const cudaError_t e = allow_smem(kern, smem, *allowed);
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
cudaError_t launch_tiles(const ShrinkParams& p, int clusters, cudaStream_t s)
{
    static std::atomic<uint64_t> allowed{0};
    return launch(shrink_tiles_kernel<BF16, RS>, tiles_smem(RS), &allowed, p, clusters, s);
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
    // A row's own cluster reads its A for itself: rows of one adapter read it again, from L2.
    const bool rows = a.M * a.K * ad.r <= (int64_t)16 << 20;
    p.work = rows ? p.M : (p.M + ROWS - 1) / ROWS;
    // K is shared by as many CTAs as fit at once and have some 256 of it.  (8192 rows of 4096: 128 tiles by two
    // CTAs each; by four, which is more than fit, FOUR)
    p.cluster = 1;
    const int fit = (rows ? 4 : 2) * num_sms;
    while (p.cluster < MAX_CLUSTER && 2 * p.cluster * p.work <= fit && 2 * p.cluster * 256 <= p.K) p.cluster *= 2;
    // (B is looked through beside the rest, by a CTA an SM)
    const int clusters = p.work + (p.lists > 0 ? (p.lists + num_sms + p.cluster - 1) / p.cluster : 0);
    cudaError_t e;
    if (rows) {
        e = a.bf16 ? launch(shrink_rows_kernel<true>, 0, nullptr, p, clusters, stream)
                   : launch(shrink_rows_kernel<false>, 0, nullptr, p, clusters, stream);
    } else {
        const auto tiles = a.bf16 ? (p.rs == 16   ? launch_tiles<true, 16>
                                     : p.rs == 32 ? launch_tiles<true, 32>
                                     : p.rs == 64 ? launch_tiles<true, 64>
                                                  : launch_tiles<true, 128>)
                                  : (p.rs == 16   ? launch_tiles<false, 16>
                                     : p.rs == 32 ? launch_tiles<false, 32>
                                     : p.rs == 64 ? launch_tiles<false, 64>
                                                  : launch_tiles<false, 128>);
        e = tiles(p, clusters, stream);
    }
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

}  // namespace gemm_gb300
