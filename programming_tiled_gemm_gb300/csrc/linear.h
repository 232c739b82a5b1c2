// Internal interface of the linear-layer kernels: products with fused epilogues, dense or
// grouped by expert, their gradients, and the routing kernels around them (not installed).
#pragma once

#include <atomic>

#include "internal.h"

namespace gemm_gb300 {

constexpr int kMaxGroups = 1024;  // the kernels keep two words a group in shared memory

// What the tensor-core kernel of linear_tc.cu computes: D[t][f] = sum_k A[f][k] B[t][k],
//   kLinFwd  Y = act(X W + b) + R    f: columns of W, t: rows of X,    reduced over K
//   kLinDx   dX = dZ W^T             f: rows of W,    t: rows of dZ,   reduced over Nw
//   kLinDw   dW = X^T dZ             f: columns of W, t: columns of X, reduced over the rows
enum LinMode { kLinFwd = 0, kLinDx = 1, kLinDw = 2 };

// Low-rank adapters beside a forward product: row m adds s_i (X[m] A_i) B_i, i = adapters[m].
constexpr int kMaxAdapterRank = 128;
constexpr int kMaxAdapters = 8192;     // (which of them are used: a bit each in shared memory)
constexpr int64_t kMaxAdaptedK = 16384;  // (one accumulator over all of K)
// (adapters.cu looks at up to 4096 row numbers past the last, in 32 bits)
constexpr int64_t kMaxAdaptedRows = ((int64_t)1 << 31) - (1 << 17);
constexpr int kAdapterParts = 32;      // of a used adapter's B, which have a byte of `bad` each
struct LinAdapt {
    int n, r, rs;  // adapters, their rank, and the rank to 16, 32, 64 or 128: a row's length in `u`
    const void* A;  // [n][K][r]
    int64_t lda, a_stride;
    const void* B;  // [n][r][Nw]
    int64_t ldb, b_stride;
    const int32_t* adapters;  // [M]; outside 0 .. n - 1: the row has none
    const float* scales;      // [n] or null: ones
    // made by launch_shrink for the product
    uint16_t* u;       // [M][rs]: s_i X A_i of the rows that have an adapter
    int* tiles;        // the row tiles' lists of adapters (adapter_list_words(rows) words each)
    uint16_t* slot;    // [M]: the row's adapter's place in its tile's list, or 0xffff
    uint8_t* bad;      // [n][kAdapterParts]: whether a used adapter's B holds infinities or NaN
    int tile_rows;     // of the product's row tiles; 0: the few-row kernel, which needs none of the last three
};
inline int adapter_list_words(int tile_rows) { return 1 + tile_rows; }

struct LinArgs {
    int mode;
    int64_t M, K, N, Nw;  // N outputs a row, Nw columns of W (2 N when gated)
    const void* X;        // kLinFwd, kLinDw: [M][K]
    int64_t ldx;
    const void* W;        // kLinFwd, kLinDx: [G][K][Nw]
    int64_t ldw, w_stride;
    const void* dZ;       // kLinDx, kLinDw: [M][Nw]
    int64_t lddz;
    const void* bias;     // [G][Nw] or null
    const void* R;        // [M][N] of the output's type or null
    int64_t ldr;
    void* Z;              // [M][Nw] or null: X W + b before the activation
    int64_t ldz;
    void* out;            // Y [M][N], dX [M][K] or dW [G][K][Nw]
    int64_t ldo, out_stride;
    int act;              // gemm_act_t
    bool bf16;            // 16-bit type of the operands
    bool out_f32;         // output (and R) in fp32 instead of that type
    int G;                // groups, or 0: one group of all rows
    const int32_t* offsets;  // device, [G + 1]: rows of group g are [offsets[g], offsets[g+1])
    // kLinDx, or null: db [G][Nw] is added up here from the pieces' sums (launch_linear_act)
    float* db;
    const float* db_ws;
    int db_piece;
    const LinAdapt* adapt;  // kLinFwd without groups, or null
};

// Forward products of a few rows without groups stream W through a kernel of their own.
bool linear_is_few(const LinArgs& a);
int launch_linear_few(const LinArgs& a, int num_sms, cudaStream_t stream, int* launches);

// Buffers the handle keeps for the linear kernels.
struct LinWorkspace {
    float* partials = nullptr;    // K slices of the last wave's tiles
    unsigned* counters = nullptr;  // arrivals; every launch leaves them zero, one that gave up as well
};

// Workspace bytes of the K-sliced last wave, and counters (of 4 bytes).
size_t linear_partials_bytes(const LinArgs& a, int num_sms, int kc);
int64_t linear_counters(int num_sms);
// Lets `kern` have `bytes` of shared memory on the current device: asked for once a device (`done`
// has a bit for each), as it takes 0.4 us of a call.  `all`: the SM's whole memory is laid out for sharing,
// so that another kernel's CTAs find room beside this one's.
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t>& done, bool all = false)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && all)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

// Returns GEMM_OK or a negative gemm_status_t.
int launch_linear(const LinArgs& a, const LinWorkspace& ws, int num_sms, int* dev_status, uint64_t limit_ns, int kc,
                  int test_stall, cudaStream_t stream, int* launches);

// The same with adapters (16-bit results, K up to 16384), whose part is there once launch_shrink's kernel
// before it has run.  The rows of its tiles, for LinAdapt::tile_rows.
int linear_tile_rows(const LinArgs& a, int num_sms);
int launch_linear_adapted(const LinArgs& a, const LinWorkspace& ws, int num_sms, int* dev_status, uint64_t limit_ns,
                          int test_stall, cudaStream_t stream, int* launches);
int launch_shrink(const LinArgs& a, const LinAdapt& ad, int num_sms, cudaStream_t stream, int* launches);

// dZ = dY act'(Z) and db = column sums of dZ, per group.
struct LinActArgs {
    int64_t M, N;
    const void* dY;
    int64_t lddy;
    const void* Z;  // [M][N], or [M][2 N] gated; unread without activation
    int64_t ldz;
    void* dZ;       // as Z; null: only db is wanted (no activation)
    int64_t lddz;
    float* db;      // [G][N or 2 N] or null
    int act;
    bool bf16;
    int G;
    const int32_t* offsets;
};
size_t linear_act_ws_bytes(const LinActArgs& a, int num_sms);
int linear_act_piece(const LinActArgs& a, int num_sms);  // rows of a piece
// `leave_sums`: the pieces' sums stay in `ws` for the dX product to add
int launch_linear_act(const LinActArgs& a, float* ws, bool leave_sums, int num_sms, cudaStream_t stream,
                      int* launches);
// Whether the dX product `a` has the time to add db's pieces of `piece` rows.
bool linear_adds_db(const LinArgs& a, int piece, int num_sms, int kc);

// First unit of every group when each group's rows are cut into pieces of `unit` rows (at
// least `least` of them) and every piece counts `per` units: cum[g] for g = 0 .. G, and the
// rows' clamped bounds in off[0 .. G].  unit = 0: `per` units a group whatever its rows.
// Every thread of the block calls it; `cum` and `off` are shared memory, read after the
// caller's next block barrier.  Offsets are clamped to [0, M] and to their running maximum,
// so that wrong ones give wrong results but no access outside the operands.
__device__ __forceinline__ int group_units(int rows, int unit, int per, int least)
{
    if (unit == 0) return per;
    return max((max(rows, 0) + unit - 1) / unit, least) * per;
}

__device__ __forceinline__ void group_table(const int32_t* offsets, int G, int M, int unit, int per, int least,
                                            int* off, int* cum)
{
    if (!offsets) {
        if (threadIdx.x == 0) {
            off[0] = 0, off[1] = M;
            cum[0] = 0, cum[1] = group_units(M, unit, per, least);
        }
        return;
    }
    for (int g = threadIdx.x; g <= G; g += blockDim.x) off[g] = min(max(offsets[g], 0), M);
    __syncthreads();
    if (threadIdx.x < 32) {
        int high = 0;
        for (int g0 = 0; g0 <= G; g0 += 32) {
            const int g = g0 + (int)threadIdx.x;
            int m = max(g <= G ? off[g] : 0, high);
#pragma unroll
            for (int d = 1; d < 32; d *= 2) m = max(m, __shfl_up_sync(0xffffffffu, m, d));
            if (g <= G) off[g] = m;
            high = __shfl_sync(0xffffffffu, m, 31);
        }
        __syncwarp();
        int base = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + (int)threadIdx.x;
            const int n = g < G ? group_units(off[g + 1] - off[g], unit, per, least) : 0;
            int s = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int u = __shfl_up_sync(0xffffffffu, s, d);
                if ((int)threadIdx.x >= d) s += u;
            }
            if (g < G) cum[g] = base + s - n;
            base += __shfl_sync(0xffffffffu, s, 31);
        }
        if (threadIdx.x == 0) cum[G] = base;
    }
}

}  // namespace gemm_gb300
