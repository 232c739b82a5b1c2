// Linear layers of a few rows (tokens): act(X W + b) + R for up to 8 rows, W streamed once.
//
// Bound by W's bytes, and for small W by latency: the tensor-core kernel's set-up, first
// loads and drain cost 5 us whatever its size.  Here a thread loads 16 bytes (eight columns) of
// eight rows of W at a time (four for more than four rows of X), all in flight, and adds their
// products with the rows of X in fp32 (packed FMAs, two columns each).  A warp covers 64
// columns x 32 (16) of K.  A CTA holds 64
// columns (gated: 32 of the gate and the 32 of the up half that belong to them); a cluster of
// up to 8 CTAs shares K and adds its sums through distributed shared memory, in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear.h"
#include "linear_math.h"
#include "ptx.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(linear_few)

namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int COLS = 64;    // columns of W a CTA
constexpr int MAX_CLUSTER = 8;

// By the registers they take: rows of W a thread has in flight, and CTAs an SM.
constexpr int deep(int rows) { return rows <= 4 ? 8 : 4; }
constexpr int resident(int rows) { return rows <= 2 ? 3 : 2; }
constexpr int batch(int rows) { return 4 * deep(rows); }  // of K, a warp

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

// The first n of eight 16-bit values, zeros for the others.
__device__ __forceinline__ uint4 first_of_8(const uint16_t* p, int n)
{
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : 0u;
    return make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16);
}

// read once: not kept in L1
__device__ __forceinline__ uint4 load_once(const uint16_t* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <bool BF16>
__device__ __forceinline__ float2 two(uint32_t u)
{
    if (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}

template <int MT, bool GATED, bool BF16>
__global__ void __launch_bounds__(THREADS, resident(MT)) linear_few_kernel(FewParams p)
{
    constexpr int OUT = GATED ? COLS / 2 : COLS, DEEP = deep(MT), BATCH = batch(MT);
    __shared__ float red[WARPS][MT * COLS];
    __shared__ float part[MT * COLS];
    grid_dependency_wait();
    grid_dependents_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = p.cluster, rank = blockIdx.x % C, out0 = blockIdx.x / C * OUT;
    // eight columns of W: of the 64, or of the gate's 32, then the up half's
    const int cl = lane % 8, kr = lane / 8;
    const int first = out0 + (GATED ? cl % 4 : cl) * 8;
    const int ncol = p.N - first;
    const uint16_t* W = p.W + first + (GATED && cl >= 4 ? p.N : 0);
    float2 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = make_float2(0.f, 0.f);
    const int batches = (p.K + BATCH - 1) / BATCH;
    for (int b = rank * WARPS + warp; b < batches; b += C * WARPS) {
        const int k0 = b * BATCH + kr * DEEP;
        uint4 w[DEEP];
        uint32_t x[MT][DEEP / 2];
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            w[u] = make_uint4(0, 0, 0, 0);
            if (k0 + u < p.K) {
                const uint16_t* row = W + (int64_t)(k0 + u) * p.ldw;
                if (ncol >= 8) w[u] = load_once(row);
                else if (ncol > 0) w[u] = first_of_8(row, ncol);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (m < p.M && k0 < p.K) {
                const uint16_t* row = p.X + m * p.ldx + k0;
                if (k0 + DEEP > p.K) v = first_of_8(row, p.K - k0);
                else if (DEEP == 8) v = *reinterpret_cast<const uint4*>(row);
                else *reinterpret_cast<uint2*>(&v) = *reinterpret_cast<const uint2*>(row);
            }
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < DEEP / 2; ++i) x[m][i] = words[i];
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            const float2 wf[4] = {two<BF16>(w[u].x), two<BF16>(w[u].y), two<BF16>(w[u].z), two<BF16>(w[u].w)};
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float2 pair = two<BF16>(x[m][u / 2]);
                const float v = u % 2 ? pair.y : pair.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = __ffma2_rn(make_float2(v, v), wf[i], acc[m][i]);
            }
        }
    }
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
        if (n >= p.N || !in_range(m, p.M)) continue;
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

template <int MT, bool GATED, bool BF16>
cudaError_t launch_typed(const FewParams& p, int blocks, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * p.cluster, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<MT, GATED, BF16>, p);
}

template <bool GATED, bool BF16>
cudaError_t launch_rows(const FewParams& p, int rows, int blocks, cudaStream_t s)
{
    if (rows == 1) return launch_typed<1, GATED, BF16>(p, blocks, s);
    if (rows == 2) return launch_typed<2, GATED, BF16>(p, blocks, s);
    if (rows == 4) return launch_typed<4, GATED, BF16>(p, blocks, s);
    return launch_typed<8, GATED, BF16>(p, blocks, s);
}

}  // namespace

bool linear_is_few(const LinArgs& a) { return a.mode == kLinFwd && a.G == 0 && a.M <= kFewRows; }

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
    const int blocks = (p.N + out - 1) / out, batches = (p.K + batch(rows) - 1) / batch(rows);
    // K is shared by as many CTAs as fit at once and have a batch for each of their warps
    int c = num_sms * resident(rows) / blocks;
    if (c > (batches + WARPS - 1) / WARPS) c = (batches + WARPS - 1) / WARPS;
    p.cluster = c < 1 ? 1 : c > MAX_CLUSTER ? MAX_CLUSTER : c;
    const cudaError_t e = a.bf16 ? (gated ? launch_rows<true, true>(p, rows, blocks, stream)
                                          : launch_rows<false, true>(p, rows, blocks, stream))
                                 : (gated ? launch_rows<true, false>(p, rows, blocks, stream)
                                          : launch_rows<false, false>(p, rows, blocks, stream));
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

}  // namespace gemm_gb300
