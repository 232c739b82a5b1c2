// Linear layers of a few rows (tokens): act(X W + b) + R for up to 8 rows, W streamed once.
//
// Bound by W's bytes, and for small W by latency: the tensor-core kernel's set-up, first
// loads and drain cost 5 us whatever its size.  Here a thread copies 16 bytes (eight columns) of
// eight rows of W a stage into slots of its own in shared memory, three stages ahead, and
// multiplies them with the rows of X in fp32 (packed FMAs, two columns each); no block barrier
// until the end.  A warp covers 64 columns x 32 of K.  A CTA holds 64 columns (gated: 32 of
// the gate and the 32 of the up half that belong to them); a cluster of up to 8 CTAs shares K
// and adds its sums through distributed shared memory, in order.
// ADAPT: a low-rank adapter of each row's choice, U = s_i X A_i from the kernel before (adapters.cu).
// Behind the batches of X and W come those of U and the rows' B, `rank` of K for every row, which count for
// that row only.  The kernel starts as that one's dependent and waits for it before it copies U.
// One row, 2048 x 2048, rank 16: 6.8 us with U's kernel (4.1 without an adapter).
// Measured (bf16, one row): 2048 x 64 2.5 us, 2048 x 2048 4.0 (tensor-core kernel 8.4 and 9.6),
// 4096 x 4096 7.4 (12.7), 8192 x 8192 23.3, 5.8 TB/s (27.3).  Dropped: loads kept in registers
// instead of the ring (4096 x 4096 12.8, and 100 us for 4 rows of 8192 x 28672); three CTAs of two
// stages an SM (8192 x 28672 75 instead of 77, 4096 x 4096 8.3 instead of 7.4).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear.h"
#include "linear_math.h"
#include "ptx.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(linear_few)

namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int MAX_ROWS = 8;
constexpr int COLS = 64;    // columns of W a CTA
constexpr int MAX_CLUSTER = 8;

constexpr int DEEP = 8;          // rows of W of a thread in a stage
constexpr int BATCH = 4 * DEEP;  // of K, a warp and stage
constexpr int STAGES = 3;
constexpr int RESIDENT = 2;      // CTAs an SM, by their shared memory

// A warp's stage: [row][lane] 16 bytes of W, then [row of X][4] 16 bytes.
constexpr int stage_bytes(int rows) { return DEEP * 512 + rows * 64; }
constexpr int smem_bytes(int rows) { return WARPS * STAGES * stage_bytes(rows); }

struct FewParams {
    int M, K, N, Nw;
    const uint16_t* X;
    int64_t ldx;
    const uint16_t* W;
    int64_t ldw;
    const uint16_t* bias;
    const void* R;
    int64_t ldr;
    uint16_t* Z;
    int64_t ldz;
    void* out;
    int64_t ldo;
    int act, out_f32, cluster;
};

struct FewAdapt {
    const uint16_t* u;  // [M][rs]
    int rs, r, n;
    const uint16_t* B;  // [n][r][Nw]
    int64_t ldb, b_stride;
    const int32_t* adapters;
};

// 16 bytes to shared memory, of which the first n (of 16-bit values, 0 .. 8) are read and the
// others zero.
__device__ __forceinline__ void copy_8(uint32_t dst, const uint16_t* src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(2 * n) : "memory");
}

template <bool BF16>
__device__ __forceinline__ float2 two(uint32_t u)
{
    if (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}

template <int MT, bool GATED, bool BF16, bool ADAPT>
__global__ void __launch_bounds__(THREADS, RESIDENT) linear_few_kernel(FewParams p, FewAdapt ad)
{
    constexpr int OUT = GATED ? COLS / 2 : COLS;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float part[MT * COLS];
    if (!ADAPT) grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = p.cluster, rank = blockIdx.x % C, out0 = blockIdx.x / C * OUT;
    // eight columns of W: of the 64, or of the gate's 32, then the up half's
    const int cl = lane % 8, kr = lane / 8;
    const int first = out0 + (GATED ? cl % 4 : cl) * 8;
    const int ncol = max(0, min(8, p.N - first));
    const int wcol = ncol > 0 ? first + (GATED && cl >= 4 ? p.N : 0) : 0;
    const uint16_t* W = p.W + wcol;
    float2 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = make_float2(0.f, 0.f);
    const int base = (p.K + BATCH - 1) / BATCH, step = C * WARPS;
    const int batches = base + (ADAPT ? (p.M * ad.r + BATCH - 1) / BATCH : 0);
    uint8_t* mine = ring + warp * STAGES * stage_bytes(MT);
    // every lane copies what it multiplies itself of W; lane (kr, m) row m's eight values of X
    const auto fetch = [&](int b, int s) {
        if (ADAPT && b >= base && b < batches) {
            // eight of K of one row's adapter
            const uint32_t at = smem_u32(mine + s * stage_bytes(MT));
            const int k = (b - base) * BATCH + kr * DEEP, m = k / ad.r, k0 = k - m * ad.r;
            const int id = m < p.M ? __ldcg(ad.adapters + m) : -1;
            const bool on = id >= 0 && id < ad.n && (ncol == 0 || in_range(wcol + ncol - 1, p.Nw));
            const uint16_t* B = ad.B + (on ? id * ad.b_stride + (int64_t)k0 * ad.ldb + wcol : 0);
#pragma unroll
            for (int u = 0; u < DEEP; ++u) copy_8(at + u * 512 + lane * 16, B + (on ? u * ad.ldb : 0), on ? ncol : 0);
            grid_dependency_wait();
            if (cl < MT) copy_8(at + DEEP * 512 + (cl * 4 + kr) * 16, ad.u + (on ? m * ad.rs + k0 : 0), on && cl == m ? 8 : 0);
        } else if (b < base) {
            const uint32_t at = smem_u32(mine + s * stage_bytes(MT));
            const int k0 = b * BATCH + kr * DEEP;
#pragma unroll
            for (int u = 0; u < DEEP; ++u) {
                const bool in = k0 + u < p.K && (ncol == 0 || (in_range(k0 + u, p.K) && in_range(wcol + ncol - 1, p.Nw)));
                copy_8(at + u * 512 + lane * 16, W + (in ? (int64_t)(k0 + u) * p.ldw : 0), in ? ncol : 0);
            }
            if (cl < MT) {
                int n = cl < p.M ? max(0, min(8, p.K - k0)) : 0;
                if (n > 0 && (!in_range(cl, p.M) || !in_range(k0 + n - 1, p.K))) n = 0;
                copy_8(at + DEEP * 512 + (cl * 4 + kr) * 16, p.X + (n > 0 ? cl * p.ldx + k0 : 0), n);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int next = rank * WARPS + warp;  // the batch to fetch
#pragma unroll
    for (int s = 0; s < STAGES; ++s, next += step) fetch(next, s);
    int s = 0;
    for (int b = rank * WARPS + warp; b < batches; b += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();
        const uint4* w = reinterpret_cast<const uint4*>(mine + s * stage_bytes(MT)) + lane;
        const uint4* xs = reinterpret_cast<const uint4*>(mine + s * stage_bytes(MT) + DEEP * 512) + kr;
        const int row = ADAPT && b >= base ? ((b - base) * BATCH + kr * DEEP) / ad.r : -1;  // whose adapter's batch it is
        uint32_t x[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint4 v = xs[m * 4];
            x[m][0] = v.x, x[m][1] = v.y, x[m][2] = v.z, x[m][3] = v.w;
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            const uint4 v = w[u * 32];
            const float2 wf[4] = {two<BF16>(v.x), two<BF16>(v.y), two<BF16>(v.z), two<BF16>(v.w)};
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (ADAPT && m != row && row >= 0) continue;  // (another row's adapter: not even its NaN)
                const float2 pair = two<BF16>(x[m][u / 2]);
                const float f = u % 2 ? pair.y : pair.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = __ffma2_rn(make_float2(f, f), wf[i], acc[m][i]);
            }
        }
        __syncwarp();
        fetch(next, s);
        next += step;
        if (++s == STAGES) s = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ADAPT) grid_dependency_wait();  // (a CTA without such a batch too: the kernel before has ended when this one has)
    __syncthreads();  // the ring is free
    float(*red)[MT * COLS] = reinterpret_cast<float(*)[MT * COLS]>(ring);
    // the warp's four parts of K, then the warps' and the cluster's sums in order
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 v = acc[m][i];
#pragma unroll
            for (int d = 8; d < 32; d *= 2) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
            }
            if (kr == 0) *reinterpret_cast<float2*>(&red[warp][m * COLS + cl * 8 + 2 * i]) = v;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < MT * COLS; e += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += red[w][e];
        part[e] = s;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    const auto total = [&](int e) {
        if (C == 1) return part[e];
        const uint32_t at = smem_u32(&part[e]);
        float t[MAX_CLUSTER];
#pragma unroll
        for (int r = 0; r < MAX_CLUSTER; ++r)
            if (r < C) t[r] = ld_shared_cluster_f32(mapa_shared(at, r));
        float s = t[0];
#pragma unroll
        for (int r = 1; r < MAX_CLUSTER; ++r)
            if (r < C) s += t[r];
        return s;
    };
    for (int e = rank * THREADS + threadIdx.x; e < p.M * OUT; e += C * THREADS) {
        const int m = e / OUT, j = e % OUT, n = out0 + j;
        if (n >= p.N || !in_range(m, p.M) || !in_range(n, p.N) || !in_range(GATED ? p.N + n : n, p.Nw)) continue;
        float v[1] = {total(m * COLS + j)};
        if (p.bias) v[0] += from_16<BF16>(p.bias[n]);
        uint16_t* z = p.Z ? p.Z + m * p.ldz + n : nullptr;
        if (z) *z = to_16<BF16>(v[0]);
        if constexpr (GATED) {
            float up = total(m * COLS + OUT + j);
            if (p.bias) up += from_16<BF16>(p.bias[p.N + n]);
            if (z) z[p.N] = to_16<BF16>(up);
            v[0] = silu(v[0]) * up;
        } else {
            activate(v, p.act);
        }
        if (p.out_f32) {
            if (p.R) v[0] += static_cast<const float*>(p.R)[m * p.ldr + n];
            static_cast<float*>(p.out)[m * p.ldo + n] = v[0];
        } else {
            if (p.R) v[0] += from_16<BF16>(static_cast<const uint16_t*>(p.R)[m * p.ldr + n]);
            static_cast<uint16_t*>(p.out)[m * p.ldo + n] = to_16<BF16>(v[0]);
        }
    }
    if (C > 1) cluster_sync_all();  // (nobody leaves while its sums are read)
}

template <int MT, bool GATED, bool BF16, bool ADAPT>
cudaError_t launch_typed(const FewParams& p, const FewAdapt& ad, int blocks, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * p.cluster, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = s;
    cfg.dynamicSmemBytes = smem_bytes(MT);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(linear_few_kernel<MT, GATED, BF16, ADAPT>, smem_bytes(MT), allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<MT, GATED, BF16, ADAPT>, p, ad);
}

template <bool GATED, bool BF16, bool ADAPT>
cudaError_t launch_rows(const FewParams& p, const FewAdapt& ad, int rows, int blocks, cudaStream_t s)
{
    if (rows == 1) return launch_typed<1, GATED, BF16, ADAPT>(p, ad, blocks, s);
    if (rows == 2) return launch_typed<2, GATED, BF16, ADAPT>(p, ad, blocks, s);
    if (rows == 4) return launch_typed<4, GATED, BF16, ADAPT>(p, ad, blocks, s);
    return launch_typed<8, GATED, BF16, ADAPT>(p, ad, blocks, s);
}

template <bool ADAPT>
cudaError_t launch_form(const LinArgs& a, const FewParams& p, const FewAdapt& ad, int rows, int blocks, cudaStream_t s)
{
    const bool gated = a.act == GEMM_ACT_SWIGLU;
    return a.bf16 ? (gated ? launch_rows<true, true, ADAPT>(p, ad, rows, blocks, s)
                           : launch_rows<false, true, ADAPT>(p, ad, rows, blocks, s))
                  : (gated ? launch_rows<true, false, ADAPT>(p, ad, rows, blocks, s)
                           : launch_rows<false, false, ADAPT>(p, ad, rows, blocks, s));
}

}  // namespace

// One row costs W's bytes alone; more are bound by the FMAs in time, and large W are then as fast
// or faster on the tensor cores.  3 rows run the kernel of 4, 5 to 7 that of 8, each at its
// time (bf16; every row count was timed).  us here and on the tensor cores, K x columns of W:
//                         1 row       2           3, 4        5 to 8
//   2048 x 2048           4.4   9.4   4.6   9.4   5.2   9.4   6.3   9.4
//   4096 x 4096           7.7  12.9   8.1  12.9   9.1  12.8  11.6  12.8
//   16384 x 1024          9.5  13.7  10.7  13.7  13.4  13.7  19.0  13.7
//   4096 x 8192          12.9  17.4  13.5  17.5  14.5  17.5  19.7  17.5
//   8192 x 8192          23.2  27.4  24.5  27.4  25.6  27.4  34.8  27.4
//   4096 x 16384 gated   22.5  24.2  24.1  24.3  27.4  24.3  36.0  24.3
//   4096 x 28672         40.1  41.5  40.0  41.6  39.7  41.6  50.7  41.8
//   8192 x 16384         44.3  42.6  46.1  42.9  46.6  42.8  64.5  42.9
//   8192 x 28672         76.7  74.4  77.1  74.4  76.3  74.5  95.3  74.8
// The limits are of W's size alone: beside them the kernel not chosen is up to 8 % faster for
// one or two rows, 11 % for three or four; for five to eight, 11 % where K is short and a third at
// 16384 x 1024, where 128 CTAs leave a part of the FMAs idle.
bool linear_is_few(const LinArgs& a)
{
    if (a.mode != kLinFwd || a.G != 0) return false;
    return a.M <= MAX_ROWS && a.K * a.Nw <= (int64_t)1 << (a.M <= 2 ? 27 : a.M <= 4 ? 26 : 24);
}

int launch_linear_few(const LinArgs& a, int num_sms, cudaStream_t stream, int* launches)
{
    const bool gated = a.act == GEMM_ACT_SWIGLU;
    FewParams p = {};
    p.M = (int)a.M, p.K = (int)a.K, p.N = (int)a.N, p.Nw = (int)a.Nw;
    p.X = static_cast<const uint16_t*>(a.X), p.ldx = a.ldx;
    p.W = static_cast<const uint16_t*>(a.W), p.ldw = a.ldw;
    p.bias = static_cast<const uint16_t*>(a.bias);
    p.R = a.R, p.ldr = a.ldr;
    p.Z = static_cast<uint16_t*>(a.Z), p.ldz = a.ldz;
    p.out = a.out, p.ldo = a.ldo;
    p.act = a.act, p.out_f32 = a.out_f32 ? 1 : 0;
    const int out = gated ? COLS / 2 : COLS, rows = p.M == 1 ? 1 : p.M == 2 ? 2 : p.M <= 4 ? 4 : 8;
    const int blocks = (p.N + out - 1) / out, batches = (p.K + BATCH - 1) / BATCH;
    // K is shared by as many CTAs as fit at once and have a batch for each of their warps
    // (clusters of 7 left GPCs half empty: 12.8 instead of 10.1 us at 4096 x 4096)
    p.cluster = 1;
    while (p.cluster < MAX_CLUSTER && 2 * p.cluster * blocks <= RESIDENT * num_sms &&
           2 * p.cluster * WARPS <= batches + WARPS - 1)
        p.cluster *= 2;
    FewAdapt ad = {};
    if (a.adapt) {
        const LinAdapt& l = *a.adapt;
        ad = {l.u, l.rs, l.r, l.n, static_cast<const uint16_t*>(l.B), l.ldb, l.b_stride, l.adapters};
    }
    const cudaError_t e = a.adapt ? launch_form<true>(a, p, ad, rows, blocks, stream)
                                  : launch_form<false>(a, p, ad, rows, blocks, stream);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

}  // namespace gemm_gb300
