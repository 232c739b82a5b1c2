// The elementwise half of a linear layer's gradient: dZ = dY act'(Z), rounded once to the
// operands' 16-bit type for the two products that follow, and db = sum over the rows of dZ
// (per group), summed in fp32 from the unrounded dZ in the same pass.
//
// Bound by memory: dY and Z are read and dZ written once, 16 bytes a thread.  Resident blocks
// walk pieces of 256 columns (a warp a row, eight columns a lane) x 8 .. 32 rows with four
// rows' loads in flight a warp, keep a piece's column sums in registers and leave them in
// the workspace.  A group's pieces are added in order by a warp of the dX product that has
// nothing else to do, or, where dX is not wanted or too short for it, by a second, small
// launch: the same sums in the same order.  (Adding them in the block that counts last took 10
// us more at 4096 x 4096: one block reads what many can.)
// 4096 x 4096 bf16: relu 15 us (6.7 TB/s), gelu_tanh 19 us (its arithmetic: over half the
// issue slots), swiglu 26 us (168 MB); with db 5 us more.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear.h"
#include "ptx.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(linear_act)

namespace {

constexpr int THREADS = 256, WARPS = 8, COLS = 256;

struct ActParams {
    int M, N, G;
    const int32_t* offsets;
    const void* dY;
    int64_t lddy;
    const void* Z;
    int64_t ldz;
    void* dZ;  // null: not wanted (no activation)
    int64_t lddz;
    float* db;  // [G][Nw] or null
    float* ws;  // [item][Nw]
    int act, col_blocks;
    int piece, items;  // rows of a piece; pieces (an upper bound over groups)
};

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t u)
{
    if (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u));
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack(float a, float b)
{
    if (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

// Eight 16-bit values of a row from element `at` on, of which the first `n` exist; as they
// are in memory, and in fp32.
__device__ __forceinline__ uint4 load8(const void* base, int64_t at, int n)
{
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (n >= 8) return __ldcs(reinterpret_cast<const uint4*>(p));  // (read once: out of L2 before dZ)
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : 0u;
    return make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16);
}

template <bool BF16>
__device__ __forceinline__ void widen(uint4 u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack<BF16>(w[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void store8(void* base, int64_t at, int n, uint4 u)
{
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if (n >= 8) {
        *reinterpret_cast<uint4*>(p) = u;
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&v)[8])
{
    store8(base, at, n, make_uint4(pack<BF16>(v[0], v[1]), pack<BF16>(v[2], v[3]), pack<BF16>(v[4], v[5]),
                                   pack<BF16>(v[6], v[7])));
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// dz[i] = dy[i] act'(z[i])
__device__ __forceinline__ void act_grad(float (&dz)[8], const float (&z)[8], int act)
{
    switch (act) {
    case GEMM_ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) dz[i] = z[i] > 0.f ? dz[i] : 0.f;
        break;
    case GEMM_ACT_GELU:  // Phi(z) + z phi(z)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dz[i] *= 0.5f * (1.f + erff(z[i] * 0.70710678118654752f)) +
                     z[i] * 0.39894228040143268f * __expf(-0.5f * z[i] * z[i]);
        break;
    case GEMM_ACT_GELU_TANH:  // s = 1 / (1 + e^-2u), 2 u = z (c + c a z^2): s + z s (1 - s) 2 u'
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float z2 = fminf(z[i] * z[i], 1e4f);  // (saturated long before; 0 times infinity is NaN)
            const float s = sigmoid(z[i] * (1.5957691216057308f + 0.07135481627260025f * z2));
            dz[i] *= s + z[i] * s * ((1.f - s) * (1.5957691216057308f + 0.2140644488178007f * z2));
        }
        break;
    case GEMM_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = sigmoid(z[i]);
            dz[i] *= s * (1.f + z[i] * (1.f - s));
        }
        break;
    default: break;
    }
}

// silu(z) u: the gate's gradient d u silu'(z) and the up half's d silu(z), q = sigmoid(z).
// (q's zero first: the other factors may overflow)
__device__ __forceinline__ void gated_grad(float d, float z, float u, float& dg, float& du)
{
    const float q = sigmoid(z), zq = z * q;
    du = d * zq;
    dg = d * (u * (q + zq * (1.f - q)));
}

template <bool BF16, bool GATED, bool BIAS>
__global__ void __launch_bounds__(THREADS, 3) linear_act_kernel(ActParams p)
{
    extern __shared__ int table[];  // off[G + 1], cum[G + 1] (BIAS)
    // a lane's eight columns lie in nine words, so that neither side meets bank conflicts
    __shared__ float sums[WARPS][32 * 9];
    constexpr int DEEP = GATED ? 2 : 4;  // rows of a warp whose loads are in flight together
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int Nw = GATED ? 2 * p.N : p.N;
    int* off = table;
    int* cum = table + p.G + 1;
    int items = p.items;
    if (BIAS) {
        group_table(p.offsets, p.G, p.M, p.piece, 1, 1, off, cum);
        __syncthreads();
        grid_dependents_launch();
        items = cum[p.G];
    }
    int g = 0;
    for (int w = blockIdx.x; w < items * p.col_blocks; w += gridDim.x) {
        const int item = w / p.col_blocks, cblock = w % p.col_blocks;
        const int col = cblock * COLS + lane * 8;
        const int ncol = p.N - col;  // columns of this lane that exist (may be <= 0 or above 8)
        int first, rows;
        if (BIAS) {
            while (cum[g + 1] <= item) ++g;  // (a block's items ascend)
            first = off[g] + (item - cum[g]) * p.piece;
            rows = min(p.piece, off[g + 1] - first);
        } else {
            first = item * p.piece;
            rows = min(p.piece, p.M - first);
        }
        if (!in_range(first, p.M + 1) || !in_range(first + rows, p.M + 1)) rows = 0;
        float s[8] = {}, su[8] = {};
        for (int r0 = warp; ncol > 0 && r0 < rows; r0 += DEEP * WARPS) {
            uint4 dy[DEEP], zg[DEEP], zu[DEEP];
#pragma unroll
            for (int i = 0; i < DEEP; ++i) {
                const int64_t row = first + r0 + i * WARPS;
                if (r0 + i * WARPS < rows) {
                    dy[i] = load8(p.dY, row * p.lddy + col, ncol);
                    if (p.dZ) zg[i] = load8(p.Z, row * p.ldz + col, ncol);
                    if (GATED) zu[i] = load8(p.Z, row * p.ldz + p.N + col, ncol);
                }
            }
#pragma unroll
            for (int i = 0; i < DEEP; ++i) {
                if (r0 + i * WARPS >= rows) break;
                const int64_t row = first + r0 + i * WARPS;
                if constexpr (GATED) {
                    // (two columns at a time, into the words they came from: registers)
                    uint32_t wd[4] = {dy[i].x, dy[i].y, dy[i].z, dy[i].w}, wu[4] = {zu[i].x, zu[i].y, zu[i].z, zu[i].w};
                    const uint32_t wz[4] = {zg[i].x, zg[i].y, zg[i].z, zg[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 d = unpack<BF16>(wd[k]), z = unpack<BF16>(wz[k]), u = unpack<BF16>(wu[k]);
                        float2 dg, du;
                        gated_grad(d.x, z.x, u.x, dg.x, du.x);
                        gated_grad(d.y, z.y, u.y, dg.y, du.y);
                        if (BIAS) s[2 * k] += dg.x, s[2 * k + 1] += dg.y, su[2 * k] += du.x, su[2 * k + 1] += du.y;
                        wd[k] = pack<BF16>(dg.x, dg.y);
                        wu[k] = pack<BF16>(du.x, du.y);
                    }
                    store8(p.dZ, row * p.lddz + col, ncol, make_uint4(wd[0], wd[1], wd[2], wd[3]));
                    store8(p.dZ, row * p.lddz + p.N + col, ncol, make_uint4(wu[0], wu[1], wu[2], wu[3]));
                } else {
                    float d[8], z[8];
                    widen<BF16>(dy[i], d);
                    if (p.dZ) {
                        widen<BF16>(zg[i], z);
                        act_grad(d, z, p.act);
                        store8<BF16>(p.dZ, row * p.lddz + col, ncol, d);
                    }
                    if (BIAS)
#pragma unroll
                        for (int k = 0; k < 8; ++k) s[k] += d[k];
                }
            }
        }
        if (!BIAS) continue;
        // the warps' sums in order, one column a thread
        float* dst = p.ws + (int64_t)item * Nw;
        const int c = cblock * COLS + threadIdx.x;
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[warp][lane * 9 + i] = h ? su[i] : s[i];
            __syncthreads();
            float t = 0.f;
#pragma unroll
            for (int q = 0; q < WARPS; ++q) t += sums[q][threadIdx.x / 8 * 9 + threadIdx.x % 8];
            if (c < p.N && in_range(item, p.items) && in_range(h * p.N + c, Nw)) dst[h * p.N + c] = t;
        }
    }
}

constexpr int SUM_WARPS = 8;

// db of 32 columns of a group: warp w adds pieces w, w + 8, ...; the warps' sums are added
// in order.  The groups' first pieces come from the same table as above.
__global__ void __launch_bounds__(32 * SUM_WARPS) linear_db_kernel(ActParams p, int Nw)
{
    extern __shared__ int table[];
    __shared__ float sums[SUM_WARPS][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int blocks = (Nw + 31) / 32, g = blockIdx.x / blocks, c = blockIdx.x % blocks * 32 + lane;
    int* cum = table + p.G + 1;
    group_table(p.offsets, p.G, p.M, p.piece, 1, 1, table, cum);
    __syncthreads();
    grid_dependency_wait();
    const float* src = p.ws + (int64_t)cum[g] * Nw + c;
    const int pieces = cum[g + 1] - cum[g];
    float t = 0.f;
    if (c < Nw && (pieces == 0 || in_range(cum[g + 1] - 1, p.items))) {
#pragma unroll 8
        for (int i = warp; i < pieces; i += SUM_WARPS) t += __ldcg(src + (int64_t)i * Nw);
    }
    sums[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < Nw && in_range(g, p.G)) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < SUM_WARPS; ++w) v += sums[w][lane];
        p.db[(int64_t)g * Nw + c] = v;
    }
}

template <bool BF16, bool GATED>
cudaError_t launch_typed(const ActParams& p, dim3 grid, cudaStream_t s)
{
    if (p.db)
        linear_act_kernel<BF16, GATED, true><<<grid, THREADS, 2 * (p.G + 1) * sizeof(int), s>>>(p);
    else
        linear_act_kernel<BF16, GATED, false><<<grid, THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

int piece_rows(const LinActArgs& a, int num_sms)
{
    const int64_t col_blocks = (a.N + COLS - 1) / COLS;
    const int64_t r = a.M * col_blocks / (3 * (int64_t)num_sms) / WARPS * WARPS;
    return (int)(r < WARPS ? WARPS : r > 32 ? 32 : r);
}

int64_t items(const LinActArgs& a, int num_sms)
{
    const int piece = piece_rows(a, num_sms);
    const int64_t n = (a.M + piece - 1) / piece;
    return a.db ? n + (a.G > 0 ? a.G : 1) : n;
}

}  // namespace

size_t linear_act_ws_bytes(const LinActArgs& a, int num_sms)
{
    return a.db ? (size_t)items(a, num_sms) * (size_t)(a.act == GEMM_ACT_SWIGLU ? 2 * a.N : a.N) * sizeof(float) : 0;
}

int linear_act_piece(const LinActArgs& a, int num_sms) { return piece_rows(a, num_sms); }

int launch_linear_act(const LinActArgs& a, float* ws, bool leave_sums, int num_sms, cudaStream_t stream,
                      int* launches)
{
    ActParams p = {};
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.G = a.G > 0 ? a.G : 1;
    p.offsets = a.G > 0 ? a.offsets : nullptr;
    p.dY = a.dY;
    p.lddy = a.lddy;
    p.Z = a.Z;
    p.ldz = a.ldz;
    p.dZ = a.dZ;
    p.lddz = a.lddz;
    p.db = a.db;
    p.ws = ws;
    p.act = a.act;
    p.col_blocks = (int)((a.N + COLS - 1) / COLS);
    const int64_t n = items(a, num_sms);
    p.piece = piece_rows(a, num_sms);
    p.items = (int)n;
    if (n == 0 || a.N == 0) return GEMM_OK;
    if (n * p.col_blocks > 0x7fff0000LL) return GEMM_ERR_UNSUPPORTED;  // (room for a stride beyond)
    const int64_t resident = 3 * (int64_t)num_sms;  // blocks walk the pieces
    const dim3 grid((unsigned)(n * p.col_blocks < resident ? n * p.col_blocks : resident));
    const bool gated = a.act == GEMM_ACT_SWIGLU;
    const cudaError_t e = a.bf16 ? (gated ? launch_typed<true, true>(p, grid, stream) : launch_typed<true, false>(p, grid, stream))
                                 : (gated ? launch_typed<false, true>(p, grid, stream) : launch_typed<false, false>(p, grid, stream));
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    if (a.db && !leave_sums) {
        const int Nw = (int)(gated ? 2 * a.N : a.N);
        const int64_t blocks = (int64_t)p.G * ((Nw + 31) / 32);
        if (blocks > 0x7fffffffLL) return GEMM_ERR_UNSUPPORTED;
        if (launch_dependent(linear_db_kernel, dim3((unsigned)blocks), dim3(32 * SUM_WARPS), 2 * (p.G + 1) * sizeof(int), stream,
                             p, Nw) != cudaSuccess)
            return GEMM_ERR_CUDA;
        *launches += 1;
    }
    return GEMM_OK;
}

}  // namespace gemm_gb300
