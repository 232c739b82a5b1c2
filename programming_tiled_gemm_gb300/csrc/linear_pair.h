// Linear layers on the 5th-generation tensor cores: the product with bias, activation and
// residual in its epilogue, for one weight matrix or for rows grouped by expert, and the
// two products of its gradient.
//
// All three are D[t][f] = sum_k A[f][k] B[t][k] with the FEATURES f on the MMA's M side and
// the ROWS t (tokens) on its N side: a CTA pair's tcgen05.mma is 256 features x w rows, and
// w is any multiple of 16 up to 256, chosen per tile at run time.  So one kernel takes a few
// tokens (w = 16: the weights stream past, nothing else counts), ragged groups (a group of
// 300 rows becomes two tiles of 160 and 140 rows instead of 512 padded ones) and large
// products (256 x 256 tiles).  Putting the features on the TMEM lanes also makes the
// epilogue's accesses contiguous: a warp holds 32 features of a row.
//   * kLinFwd: A is W (MN-major in shared memory: W is K x N row-major), B is X (K-major);
//   * kLinDx:  A is W read along N (K-major), B is dZ (K-major);
//   * kLinDw:  A is dZ, B is X, both MN-major, reduced over the rows.
// Gated (SwiGLU): W's gate columns f and up columns N + f are rows 0..63 and 64..127 of a
// CTA's operand, so a tile holds both halves of 128 outputs; the two halves lie in
// different TMEM lanes, and each pair of epilogue warps swaps half of its columns through
// shared memory.
//
// Pipeline, as in the plain product's CTA-pair kernel: TMA producers, a ring of stages, one
// warp a pair that issues MMAs, eight epilogue warps a CTA.  The tensor core's fp32
// accumulation rounds toward zero: up to 2^-23 of the PARTIAL sum is lost per 16 of K.  For fp32
// results, and for more than 16384 of K, it is cut into chunks of `kc` k-blocks (16: 1024 of K, as
// in the plain product), each in a fresh TMEM accumulator, added in fp32 round-to-nearest
// registers in order (CHUNKED).  Otherwise one accumulator takes all of K (or of a slice), and
// the epilogue, which takes its sums straight from TMEM, overlaps the whole next tile.  At 16384
// that loses 2^-13 of the largest partial sum at most, a quarter of an fp16 result's own
// rounding and 1/32 of a bf16 result's where the sum does not cancel (measured, products of one
// sign: 1.0e-4, 2^-13.2; in chunks 5.4e-6).  Sums of random signs lose far less, as their partial
// sums stay small.  Where a sum cancels, the loss is still of the large partial sum: halves that
// cancel to 1/230 were off by 3.9e-3 (fp16) and 4.1e-3 (bf16) of the result, 2.1e-4 and 1.7e-3
// in chunks, which GEMM_OPT_TC_CHUNK asks for.
//
// Work: tiles are walked round robin by the persistent pairs.  The tiles of the last,
// partial wave (all tiles, when there are fewer than pairs) may be cut along K into slices,
// one a pair.  Every slice goes to the workspace in fp32; the CTA that counts last adds the
// slices of its tile in K order and runs the epilogue.  Nothing waits for another CTA, and
// the order of the sum does not depend on who is last.  A CTA that gave up on a wait is counted
// too, so that every launch leaves the counters zero.
//
// kLinDw over groups: a group's last k-block ends inside the next group's rows.  Those rows
// are zeroed in shared memory, in both operands (zero times a neighbour's NaN would be NaN),
// by a fixer warp before the MMAs may read the stage.
//
// Measured (GB300, bf16; the plain product's measured rate is 1878 TFLOP/s, copies 6.79 TB/s):
//   8192^3, bias, gelu_tanh and residual: 575 us in a burst, 1912 TFLOP/s, tensor pipe busy;
//     (the plain product 571) and 680 to 700 us (1570 to 1620 TFLOP/s) back to back under the
//     power limit
//   4096^3: dX 74 us, dW 81 us, with the full epilogue 81 us (tensor pipe 90, 88, 81 % active)
//   16 x 8192 x 8192: 27 us, 4.9 TB/s; 16 x 8192 x 28672: 75 us, 6.3 TB/s (HBM)
//   16 x 2048 x 2048: 9.6 us, latency: 5 us of launch, set-up, first loads and drain, then
//     0.14 us a k-block or 2.5 us for a cut.  (Fewer rows: linear_few.cu)
//   16384 rows over 32 experts, 2048 x 4096 swiglu, loads of 7 to 1610 rows: 188 us; 256-row
//     tiles at 515 cycles a k-block, narrower ones bound by their loads
// Every wait is bounded; on expiry the status word is set and the CTA drains and returns.
//
// ADAPT (kLinFwd): a low-rank adapter of each row's choice, Z = X W + b + U B_i with U = s_i X A_i of
// 16 bits from the kernel before (adapters.cu).  It is a longer reduction: after a tile's last
// k-block of X and W come blocks of 64 more of K, in which the tile's adapters lie side by side, `rs` of
// K each: TMA brings their rows of B as it brings W's, and an otherwise idle warp copies the rows' U, zero
// outside the row's own adapter.  So the sum stays in one accumulator, and a tile pays one block more for four
// adapters of rank 16.  These blocks have one to four places of their own beside the ring, filled while the
// tile's own k-blocks run: in the ring, they came 4 us after the tile's last one.  The kernel starts as the
// dependent of the one that makes U and waits for it only before these blocks; X was complete before that one
// started.  Measured (bf16, both kernels): 32 x 4096 x 4096, 16 adapters of rank 16, 24 us (without adapters 14.5: U 4,
// the adapters' blocks 3, their part of the slices 2); 8192 x 4096 x 4096 swiglu, 8 adapters of rank 64, 197 us (142; U
// 30, the blocks the rest).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "linear.h"
#include "linear_math.h"
#include "ptx.h"

namespace gemm_gb300 {

namespace {

constexpr int BK = 64;                // k per stage: one 128-byte swizzle row of 16-bit values
constexpr int UMMA_K = 16;
constexpr int CTA_F = 128;            // features (MMA rows) of one CTA
constexpr int MAX_W = 256;            // rows (MMA columns) of a tile
constexpr int NARROW_W = 128;         // and with chunks, whose sums an epilogue thread holds: 64 of them
constexpr int A_BYTES = CTA_F * BK * 2;  // 16 KiB a stage
constexpr int BOX_BYTES = 64 * BK * 2;   // 64 x 64 box of an MN-major operand
constexpr int MAX_STAGES = 12;
constexpr int MAX_KB_WHOLE = 256;     // k-blocks one accumulator takes for a 16-bit result
constexpr int RASTER = 8;             // row tiles per raster group (2048 rows share W's columns in L2)
constexpr int STG_BYTES = 2048;       // an epilogue warp's staging block: 32 rows x 32 features of 16 bits,
                                      // or (gated) 16 columns of fp32 for the other warp
constexpr int SMEM_MAX = 232448;      // 227 KiB
constexpr unsigned SLICE_MISSING = 1u << 16;  // in the count of a tile's slices: one that gave up

// Warps 0..3: producer of A, MMA issuer, fixer (kLinDw; db's sums in kLinDx), producer of B; 4..11: epilogue, which takes
// registers from the first four: 80 + 2 * 208 a thread of the three warpgroups are within
// the 3 * 168 the block is launched with (checked before the launch).
constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int EPI_GROUPS = EPI_WARPS / 4;  // four warps cover the TMEM lanes
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int LAUNCH_REGS = 168, LEAN_REGS = 80, EPI_REGS = 208;
static_assert(LEAN_REGS + 2 * EPI_REGS <= 3 * LAUNCH_REGS, "the epilogue's registers come from the block's own");

struct LinParams {
    int M;       // rows of X
    int rows;    // extent of the row (t) side: M, or K for kLinDw
    int F;       // output columns
    int kb;      // k-blocks of a tile (kLinDw over groups: taken from the group's rows)
    int G;
    const int32_t* offsets;
    int f_tiles;
    int bx;      // rows of a K-major B box
    int b_bytes, stages, kc;
    unsigned per_inv;  // 2^32 / (RASTER * f_tiles), rounded down
    int wcap;        // rows of a tile at most (a multiple of 16)
    int split_w;     // tile width the last wave's split is planned for (0: no split)
    const void* bias;
    int64_t bias_stride;
    const void* R;
    int64_t ldr;
    void* Z;
    int64_t ldz;
    void* out;
    int64_t ldo, out_stride;
    int act, out_f32;
    int vec_r, vec_z, vec_out;  // 16-bit R, Z and out with 16-byte aligned rows
    uint32_t idesc;  // without N
    float* ws;
    unsigned* cnt;
    int ws_cols;     // columns of a partial tile in the workspace
    int* status;
    uint64_t limit_ns;
    int test_stall;  // test hook: pair n - 1 first waits on a barrier nothing arrives on (-1: every pair)
    float* db;       // kLinDx: [G][db_cols], the sums of the pieces of db_piece rows in db_ws, or null
    const float* db_ws;
    int db_piece, db_cols;
};

// The width of `rows` rows' tiles of at most `wcap` (a multiple of 16): equal ones, so that
// 300 rows are 160 + 140, not 256 + 44.  (kLinDw: wcap itself.  Its rows lie along a line of
// X, and copies from the middle of 128-byte lines took twice the time: 1.17 ms instead of
// 0.67 at 8192^3 with 176 rows.)
__host__ __device__ inline int tile_width(int mode, int rows, int wcap)
{
    if (mode == kLinDw) return wcap;
    if (rows <= wcap) return (rows + 15) / 16 * 16;
    const unsigned nt = (unsigned)(rows + wcap - 1) / (unsigned)wcap;
    const unsigned w = ((unsigned)rows + nt - 1) / nt;
    return (int)((w + 15) / 16 * 16);
}

// Estimated cycles, fitted to measurements: a k-block of a tile of w rows (its MMAs and loads,
// or their issue: 0.14 us up to 64 rows, 0.2 us for 160, 0.26 us for 256), and what cutting a tile into S
// slices along K costs: their publication, the count and the addition, six slices' loads at a
// time (2.5 us for 2 to 6 slices of 16 rows, 4.4 us of 64, 12.8 us of 256).
constexpr int SUM_DEEP = 6;
__host__ __device__ inline int kb_cycles(int w) { return w <= 64 ? 270 : w <= 178 ? 380 : 67 + w * 7 / 4; }
__host__ __device__ inline int split_cycles(int S, int w)
{
    return S < 2 ? 0 : 3500 + w * (74 + 5 * S + 60 * ((S - 1) / SUM_DEEP));
}

// K slices of each of the last wave's `rem` tiles of kb k-blocks (1: whole), at most one a
// pair: one or two rounds of additions, where that costs less than it saves.
__host__ __device__ inline int slices(int rem, int kb, int pairs, int w)
{
    if (rem <= 0 || w <= 0) return 1;
    int best = 1;
    int64_t least = (int64_t)kb * kb_cycles(w);
    for (int round = 1; round <= 2; ++round) {
        const int S = min(min(pairs / rem, kb / 2), round * SUM_DEEP);
        if (S < 2) break;
        const int64_t t = (int64_t)((kb + S - 1) / S) * kb_cycles(w) + split_cycles(S, w);
        if (t < least) least = t, best = S;
    }
    return best;
}

struct Item {
    int g, row0, valid, w, f0;  // group, first row, rows to store, tile width, first feature
    int kb0, kb1;               // k-blocks
    int red0, red_rows;         // kLinDw: first reduced row of the group, its rows
    int part, slot0;            // slice: index among the last wave's tiles (-1: whole), the first slice's place
};

// The work items of one pair, in the order every role of the kernel walks them.  (All in 32
// bits: a 64-bit division takes hundreds of cycles.)
template <int MODE>
class Walk {
  public:
    __device__ Walk(const LinParams& p, const int* off, const int* cum, int pair, int pairs)
        : p_(p), off_(off), cum_(cum), pairs_(pairs), t_(pair), g_(0), tail_(-1)
    {
        const int total = cum[p.G];
        const int rem = total % pairs;
        whole_ = total;
        S_ = slices(rem, p.kb, pairs, p.split_w);
        if (S_ > 1) {
            whole_ = total - rem;
            if (pair < rem * S_) tail_ = pair;
        }
    }

    __device__ bool next(Item& it)
    {
        int tile;
        it.part = -1;
        if (t_ < whole_) {
            tile = t_;
            t_ += pairs_;
            it.kb0 = 0, it.kb1 = p_.kb;
        } else if (tail_ >= 0) {
            const unsigned j = (unsigned)tail_ / (unsigned)S_, sl = tail_ - j * S_;
            it.part = (int)j;
            it.slot0 = (int)j * S_;
            it.kb0 = (int)(sl * (unsigned)p_.kb / (unsigned)S_);
            it.kb1 = (int)((sl + 1) * (unsigned)p_.kb / (unsigned)S_);
            tile = whole_ + (int)j;
            slot_ = tail_;
            tail_ = -1;
        } else {
            return false;
        }
        if (tile >= end_ || w_ == 0) {
            // the next group with this tile: its rows, tiles and their width
            while (tile >= cum_[g_ + 1]) ++g_;
            begin_ = cum_[g_], end_ = cum_[g_ + 1];
            first_ = off_[g_], rows_ = off_[g_ + 1] - first_;
            const int n = MODE == kLinDw ? p_.rows : rows_;
            nt_ = (unsigned)(n + p_.wcap - 1) / (unsigned)p_.wcap;
            w_ = tile_width(MODE, n, p_.wcap);
        }
        it.g = g_;
        it.w = w_;
        int rows = rows_, first = first_;
        if (MODE == kLinDw) {
            it.red0 = first;
            it.red_rows = rows;
            if (p_.offsets) it.kb0 = 0, it.kb1 = (rows + BK - 1) / BK;
            rows = p_.rows, first = 0;
        }
        // raster: groups of RASTER row tiles, the rows fastest (division by a launch constant)
        const unsigned local = tile - begin_, per = RASTER * p_.f_tiles;
        unsigned rg = __umulhi(local, p_.per_inv);
        if (local - rg * per >= per) ++rg;
        const unsigned m0 = rg * RASTER, r = local - rg * per, m = min(nt_ - m0, (unsigned)RASTER);
        const unsigned ft = m == RASTER ? r / RASTER : r / m;
        const int t0 = (int)(m0 + r - ft * m) * it.w;
        it.row0 = first + t0;
        it.valid = min(it.w, rows - t0);
        it.f0 = (int)ft;  // (in tiles; the caller scales it)
        return true;
    }

    __device__ int slices_of_tile() const { return S_; }
    __device__ int slot() const { return slot_; }  // this slice's place in the workspace

  private:
    const LinParams& p_;
    const int* off_;
    const int* cum_;
    int pairs_, t_, g_, whole_, S_, tail_, slot_ = 0;
    int begin_ = 0, end_ = 0, first_ = 0, rows_ = 0, w_ = 0;  // the current group
    unsigned nt_ = 0;
};

__device__ __forceinline__ void record_error(int* status, int code, volatile int* abort_flag)
{
    atomicCAS(status, 0, code);
    *abort_flag = 1;
}

// The epilogue's 16-bit matrices as it reads and writes them: a warp holds 32 features (one
// a lane) of N rows, and the rows lie `ld` apart.  With 16-byte aligned rows (`vec`) the
// block goes through the warp's staging block as words of two rows, [row pair][feature]:
// a lane then holds eight features of a row pair and makes one 16-byte access a row.  The
// lanes of odd row pairs take their two halves in the other order, so that the 16-byte
// accesses to shared memory meet no bank conflicts.
struct Matrix16 {
    uint16_t* base;  // row 0, feature 0 of the block
    int ld;
    int n, nf;       // rows and features of the block that exist (nf may exceed 32)
    bool vec;
    __device__ __forceinline__ uint16_t* at(int row, int f) const { return base + (int64_t)row * ld + f; }
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack_16(float lo, float hi)
{
    if (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// eight features of one row
__device__ __forceinline__ void store_row8(const Matrix16& m, int row, int f, uint4 v)
{
    if (row >= m.n || f >= m.nf) return;
    uint16_t* o = m.at(row, f);
    if (f + 8 <= m.nf) {
        *reinterpret_cast<uint4*>(o) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (f + i < m.nf) o[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}

__device__ __forceinline__ uint4 load_row8(const Matrix16& m, int row, int f)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row >= m.n || f >= m.nf) return v;
    const uint16_t* o = m.at(row, f);
    if (f + 8 <= m.nf) return *reinterpret_cast<const uint4*>(o);
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (f + i < m.nf) w[i / 2] |= (uint32_t)o[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16, int N>
__device__ __forceinline__ void store_block(const Matrix16& m, uint32_t* stg, int lane, const float (&v)[N])
{
    if (m.n <= 0 || m.nf <= 0) return;  // (uniform over the warp)
    if (!m.vec) {
        uint16_t* o = m.base + lane;
        if (lane < m.nf)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < m.n) o[(int64_t)i * m.ld] = to_16<BF16>(v[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) stg[i * 32 + lane] = pack_16<BF16>(v[2 * i], v[2 * i + 1]);
    __syncwarp();
    // features f .. f+7 of row pairs pr, pr + 8
    const int pr = lane / 4, f = lane % 4 * 8, odd = pr & 1;
    const uint4* src = reinterpret_cast<const uint4*>(stg + pr * 32 + f);
    const bool whole = m.n >= N && m.nf >= 32;  // (uniform over the warp)
    uint16_t* o = m.at(2 * pr, f);
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
        const uint4 x = src[i * 64 + odd], y = src[i * 64 + (odd ^ 1)];
        const uint4 lo = odd ? y : x, hi = odd ? x : y;  // features f..f+3, f+4..f+7
        const uint4 even = make_uint4(__byte_perm(lo.x, lo.y, 0x5410), __byte_perm(lo.z, lo.w, 0x5410),
                                      __byte_perm(hi.x, hi.y, 0x5410), __byte_perm(hi.z, hi.w, 0x5410));
        const uint4 next = make_uint4(__byte_perm(lo.x, lo.y, 0x7632), __byte_perm(lo.z, lo.w, 0x7632),
                                      __byte_perm(hi.x, hi.y, 0x7632), __byte_perm(hi.z, hi.w, 0x7632));
        if (whole) {
            *reinterpret_cast<uint4*>(o + (int64_t)(16 * i) * m.ld) = even;
            *reinterpret_cast<uint4*>(o + (int64_t)(16 * i + 1) * m.ld) = next;
        } else {
            store_row8(m, 2 * pr + 16 * i, f, even);
            store_row8(m, 2 * pr + 16 * i + 1, f, next);
        }
    }
    __syncwarp();
}

// The residual's block as it is loaded, ahead of its use: rows 2 pr and 2 pr + 1 of each lane's
// eight features.
template <int N>
struct Ahead {
    uint4 r[N / 16][2];
    __device__ __forceinline__ void load(const Matrix16& m, int lane)
    {
        if (!m.vec) return;
        const int row = lane / 4 * 2, f = lane % 4 * 8;
        if (m.n >= N && m.nf >= 32) {
#pragma unroll
            for (int i = 0; i < N / 16; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) r[i][k] = *reinterpret_cast<const uint4*>(m.at(row + 16 * i + k, f));
        } else {
#pragma unroll
            for (int i = 0; i < N / 16; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) r[i][k] = load_row8(m, row + 16 * i + k, f);
        }
    }
};

template <bool BF16, int N>
__device__ __forceinline__ void add_block(const Matrix16& m, const Ahead<N>& a, uint32_t* stg, int lane, float (&v)[N])
{
    if (m.n <= 0 || m.nf <= 0) return;
    if (!m.vec) {
        const uint16_t* r = m.base + lane;
        if (lane < m.nf)
#pragma unroll
            for (int b = 0; b < N; b += 16) {
                uint16_t t[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (b + i < m.n) t[i] = r[(int64_t)(b + i) * m.ld];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (b + i < m.n) v[b + i] += from_16<BF16>(t[i]);
            }
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
        const int pr = i * 8 + lane / 4, f = lane % 4 * 8;
        const uint4 e = a.r[i][0], o = a.r[i][1];
        uint4* dst = reinterpret_cast<uint4*>(stg + pr * 32 + f);
        const uint4 lo = make_uint4(__byte_perm(e.x, o.x, 0x5410), __byte_perm(e.x, o.x, 0x7632),
                                    __byte_perm(e.y, o.y, 0x5410), __byte_perm(e.y, o.y, 0x7632));
        const uint4 hi = make_uint4(__byte_perm(e.z, o.z, 0x5410), __byte_perm(e.z, o.z, 0x7632),
                                    __byte_perm(e.w, o.w, 0x5410), __byte_perm(e.w, o.w, 0x7632));
        dst[pr & 1] = (pr & 1) ? hi : lo;
        dst[(pr & 1) ^ 1] = (pr & 1) ? lo : hi;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t w = stg[i * 32 + lane];
        v[2 * i] += from_16<BF16>((uint16_t)w);
        v[2 * i + 1] += from_16<BF16>((uint16_t)(w >> 16));
    }
    __syncwarp();
}

// The same in fp32: a row's 32 features are 128 contiguous bytes as they are.
template <int N>
__device__ __forceinline__ void store_f32(const float* R, int64_t ldr, float* out, int64_t ldo, int n, bool on,
                                          float (&v)[N])
{
    if (!on) return;
    if (R) {
#pragma unroll
        for (int b = 0; b < N; b += 16) {
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (b + i < n) t[i] = R[(b + i) * ldr];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (b + i < n) v[b + i] += t[i];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) out[i * ldo] = v[i];
}

// db, by one warp of every CTA: 32 columns of a group at a time.  Pieces i, i + 8, ... have a
// sum each and these are added in order, as linear_db_kernel's eight warps do; sixteen
// loads in flight.
__device__ __forceinline__ void add_db(const LinParams& p, const int* off, int lane)
{
    constexpr int SUMS = 8, FLY = 16;
    const int blocks = (p.db_cols + 31) / 32;
    int g = -1, first = 0, n = 0;  // a group, its first piece and its pieces
    for (int item = blockIdx.x; item < p.G * blocks; item += gridDim.x) {
        const int at = item / blocks, c = (item - at * blocks) * 32 + lane;
        for (; g < at; ++g) {
            first += n;
            n = group_units(off[g + 2] - off[g + 1], p.db_piece, 1, 1);
        }
        if (c >= p.db_cols) continue;
        const float* src = p.db_ws + (int64_t)first * p.db_cols + c;
        float t[SUMS] = {};
        for (int i = 0; i < n; i += FLY) {
            float u[FLY];
#pragma unroll
            for (int j = 0; j < FLY; ++j)
                if (i + j < n) u[j] = __ldcg(src + (int64_t)(i + j) * p.db_cols);
#pragma unroll
            for (int j = 0; j < FLY; ++j)
                if (i + j < n) t[j % SUMS] += u[j];
        }
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < SUMS; ++j) v += t[j];
        p.db[(int64_t)at * p.db_cols + c] = v;
    }
}

// A wait that lasts for other roles' many steps, of which each has waits of its own: the limit
// counts from the last step seen (`progress`, which moves with the tiles), not from its start, or
// it would be a limit to a healthy launch's time.
__device__ __forceinline__ bool mbar_wait_while(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag,
                                                volatile int* progress)
{
    int seen = *progress;
    while (!mbar_wait_cluster(bar, parity, limit_ns, abort_flag)) {
        const int now = *progress;
        if (now == seen || (abort_flag && *abort_flag)) return false;
        seen = now;
    }
    return true;
}

struct AdaptParams {
    const uint16_t* u;   // [M][rs]
    const int* tiles;    // [row tile][words]: how many adapters the tile has, and which
    const uint16_t* slot;  // [M]: the row's adapter's place in its tile's list, or 0xffff
    const uint8_t* bad;  // [n][kAdapterParts]: an adapter whose B holds infinities or NaN
    int rs, n, words;    // of K an adapter takes; adapters; of a tile's list
    int places;          // for blocks of 64 of K of the adapters
};
constexpr int ADAPT_SMEM = MAX_W / 2 * 2;  // the fixer's copy of its rows' slots

// KPS: k-blocks of a stage, which are waited for and committed together.
template <int MODE, bool GATED, bool BF16, bool CHUNKED, int KPS, bool ADAPT>
__device__ __forceinline__ void linear_pair_body(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmE,
                                                 const LinParams& p, const AdaptParams& ad)
{
    static_assert(!ADAPT || (MODE == kLinFwd && !CHUNKED), "adapters extend the forward product's accumulator");
    constexpr bool A_MN = MODE != kLinDx, B_MN = MODE == kLinDw;
    constexpr int TILE_F = GATED ? CTA_F : 2 * CTA_F;  // output features of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t* smem_a = smem;
    const int slots_all = p.stages * KPS + (ADAPT ? ad.places : 0);  // (the adapters' places lie behind the ring's)
    uint8_t* smem_b = smem + slots_all * A_BYTES;
    uint8_t* after = smem_b + slots_all * p.b_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(after + EPI_WARPS * STG_BYTES);
    uint64_t* full_bar = bars;                     // (used in the even CTA)
    uint64_t* empty_bar = bars + MAX_STAGES;       // (both CTAs, multicast)
    uint64_t* tail_bar = bars + 2 * MAX_STAGES;    // kLinDw: a stage the fixer passes on (each CTA's own)
    uint64_t* peer_bar = bars + 3 * MAX_STAGES;    // kLinDw: the odd CTA's fixer is done (used in the even CTA)
    uint64_t* free_bar = tail_bar;                 // ADAPT: a place's MMAs are done (both CTAs, multicast)
    uint64_t* there_bar = peer_bar;                // ADAPT: a place is filled: B by TMA, both CTAs' U (used in the even CTA)
    uint64_t* tfull_bar = bars + 4 * MAX_STAGES;   // [2] (both CTAs, multicast)
    uint64_t* tempty_bar = tfull_bar + 2;          // [2] (used in the even CTA)
    uint64_t* drain_bar = tfull_bar + 4;           // (both CTAs, multicast)
    uint64_t* never_bar = tfull_bar + 5;           // never completes (test hook)
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tfull_bar + 6);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_holder + 2);
    volatile int* progress = reinterpret_cast<volatile int*>(tmem_holder + 3);  // accumulators the epilogue has had
    int* off = reinterpret_cast<int*>(tmem_holder + 4);
    int* cum = off + p.G + 1;

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const uint16_t pair_mask = 0x3;
    const int pair = blockIdx.x / 2;
    const int npairs = gridDim.x / 2;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < (ADAPT ? max(p.stages, ad.places) : p.stages); ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
            mbar_init(smem_u32(&tail_bar[s]), 1);
            mbar_init(smem_u32(&peer_bar[s]), ADAPT ? 3 : 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull_bar[a]), 1);
            mbar_init(smem_u32(&tempty_bar[a]), 2 * EPI_WARPS);
        }
        mbar_init(smem_u32(drain_bar), 1);
        mbar_init(smem_u32(never_bar), 1);
        *abort_flag = 0;
        *progress = 0;
        mbar_fence_init();
        if (p.kb > 0) {
            prefetch_tensormap(&tmA);
            prefetch_tensormap(&tmB);
        }
        if (ADAPT) prefetch_tensormap(&tmE);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), 2 * MAX_W);
        tc_fence_before();
    }
    if (!ADAPT) grid_dependency_wait();  // what follows reads what the kernel before this one wrote
    grid_dependents_launch();
    // A tile's list of adapters: how many, then which.  It is there once the kernel before has ended, which every
    // warp that reads it waits for where it first needs it.  Later tiles' words are asked for as the tile begins.
    const auto list_at = [&](const Item& it) { return ad.tiles + (int64_t)(it.row0 / it.w) * ad.words; };
    const auto word_now = [](const int* q) {
        int v;
        asm volatile("ld.global.cg.b32 %0, [%1];" : "=r"(v) : "l"(q) : "memory");
        return v;
    };
    // Lane i's adapter first + i of a list (or -1), and that adapter's flags.
    const auto id_of = [&](const Item& it, int first) {
        const int at = 1 + first + (int)(threadIdx.x % 32);
        const int id = at < ad.words ? word_now(list_at(it) + at) : -1;
        return id >= 0 && id < ad.n ? id : -1;  // (words past the list's end are anything)
    };
    const auto flags_of = [&](int id, uint4(&f)[2]) {
        const uint8_t* q = ad.bad + (int64_t)max(id, 0) * kAdapterParts;
        asm volatile("ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(f[0].x), "=r"(f[0].y), "=r"(f[0].z), "=r"(f[0].w) : "l"(q) : "memory");
        asm volatile("ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(f[1].x), "=r"(f[1].y), "=r"(f[1].z), "=r"(f[1].w) : "l"(q + 16) : "memory");
    };
    // ad.n (which TMA reads as zeros) for an adapter whose B holds infinities or NaN: zero times these is NaN and would
    // reach every row of the tile.  Its own rows' U is then NaN.
    const auto usable = [&](int id, const uint4(&f)[2]) {
        return id < 0 || (f[0].x | f[0].y | f[0].z | f[0].w | f[1].x | f[1].y | f[1].z | f[1].w) != 0 ? ad.n : id;
    };
    if (MODE == kLinDw)
        group_table(p.offsets, p.G, p.M, 0, (p.rows + p.wcap - 1) / p.wcap * p.f_tiles, 0, off, cum);
    else
        group_table(p.offsets, p.G, p.M, p.wcap, p.f_tiles, 0, off, cum);
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    bool aborted = false;

    if (warp < EPI_WARP0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LEAN_REGS));
        if (warp == 0 || warp == 3) {
            // ---------------------------------------------------------------- producers
            // warp 0 loads A (and announces a stage's bytes), warp 3 loads B: one thread issuing
            // all of a stage's copies was what the MMAs waited for
            // (whole warps walk and one elected lane issues, as the MMA warp)
            Walk<MODE> walk(p, off, cum, pair, npairs);
            Item it;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            const bool load_a = warp == 0;
            const uint32_t a_base = smem_u32(smem_a), b_base = smem_u32(smem_b);
            const uint32_t full0 = mapa_shared(smem_u32(full_bar), 0), tail_own = mapa_shared(smem_u32(tail_bar), rank);
            const uint32_t there0 = mapa_shared(smem_u32(there_bar), 0);
            bool listed = false;  // ADAPT: the lists are there
            bool first_tile = true;
            int place = 0;  // the next block's place
            uint32_t place_phase = 0;
            while (ok && walk.next(it)) {
                const int f0 = it.f0 * TILE_F;
                const int half = it.w / 2;
                const int nb = B_MN ? (half + 63) / 64 : (half + p.bx - 1) / p.bx;
                const uint32_t b_box = B_MN ? BOX_BYTES : p.bx * 128;
                const uint32_t bytes = A_BYTES + nb * b_box;
                const int b_row = it.row0 + (int)rank * half;
                // A's two boxes of 64 features (kLinDx: one of 128 rows of W)
                const int fa = GATED ? f0 + 64 * (int)rank : f0 + CTA_F * (int)rank;
                const int fa2 = GATED ? p.F + fa : fa + 64;
                // ADAPT, warp 0: the list's words and flags are asked for ahead of their use
                const bool adapts = ADAPT && load_a && it.kb1 == p.kb;
                int count = 0, id = -1, mine = 0, block = 0, seen = 0;
                uint4 flags[2] = {};
                if (adapts && listed) count = word_now(list_at(it)), id = id_of(it, 0);
                // blocks of 64 of K of the tile's adapters, up to the `to`-th
                const auto adapter_blocks = [&](int to) {
                    const int depth = min(ad.rs, BK);
                    for (; block < to && block * BK < count * ad.rs && ok; ++block) {
                        // the adapters of these 64 of K (one of them, or a part of one, from a rank of 64 on)
                        const int k = block * BK, s0 = k / ad.rs, n = min(BK / depth, count - s0), k0 = k - s0 * ad.rs;
                        if (s0 > 0 && s0 % 32 == 0 && k0 == 0) {
                            id = id_of(it, s0);
                            flags_of(id, flags);
                        }
                        if (s0 % 32 == 0 && k0 == 0) mine = usable(id, flags);
                        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&free_bar[place]), place_phase ^ 1, p.limit_ns, abort_flag))) {
                            record_error(p.status, kDevTimeoutProducer, abort_flag);
                            ok = false;
                            break;
                        }
                        int ids[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) ids[i] = __shfl_sync(0xffffffffu, mine, (s0 + i) % 32);
                        if (elect_one()) {
                            const uint32_t bar = there0 + place * 8, dst = a_base + (p.stages * KPS + place) * A_BYTES;
                            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&there_bar[place]), 2 * n * 2 * depth * 128);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i < n) {
                                    tma_load_3d_pair(dst + i * depth * 128, &tmE, bar, fa, k0, ids[i]);
                                    tma_load_3d_pair(dst + i * depth * 128 + BOX_BYTES, &tmE, bar, fa2, k0, ids[i]);
                                }
                        }
                        __syncwarp();
                        if (++place == ad.places) {
                            place = 0;
                            place_phase ^= 1;
                        }
                    }
                };
                for (int kb = it.kb0; kb < it.kb1; kb += KPS) {
                    if (ADAPT && !load_a && it.kb1 == p.kb && seen++ == p.stages)
                        grid_dependency_wait();  // (the MMA warp does there: the next wait's limit starts behind it)
                    if (ADAPT && adapts) {
                        // Once the ring has come round, the last tile's blocks have left their places (and there is
                        // time enough until this tile's are needed).
                        if (seen == p.stages && !listed) {
                            grid_dependency_wait();
                            listed = true;
                            count = word_now(list_at(it)), id = id_of(it, 0);
                            seen = 0;
                        } else if (seen == 1 && listed) {
                            flags_of(id, flags);
                        } else if (seen == (first_tile ? 2 : p.stages) && listed) {
                            adapter_blocks(ad.places);
                        }
                        ++seen;
                    }
                    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty_bar[stage]), phase ^ 1, p.limit_ns, abort_flag))) {
                        record_error(p.status, kDevTimeoutProducer, abort_flag);
                        ok = false;
                        break;
                    }
                    // a k-block that ends inside the next group's rows goes through the fixer
                    const bool tail = MODE == kLinDw && p.offsets && it.red_rows - kb * BK < BK;
                    // (the even CTA alone announces both CTAs' bytes: arrivals from the odd one,
                    // released at cluster scope, took the kernel from 0.71 to 1.66 ms at 8192^3)
                    const uint32_t bar = (tail ? tail_own : full0) + stage * 8;
                    const int n = KPS == 1 ? 1 : min(KPS, it.kb1 - kb);
                    if (elect_one()) {
                        if (load_a) {
                            if (tail) mbar_arrive_expect_tx(smem_u32(&tail_bar[stage]), bytes);
                            else if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), 2 * n * bytes);
                        }
#pragma unroll
                        for (int i = 0; i < KPS; ++i) {
                            if (i >= n) break;
                            const int k = (MODE == kLinDw ? it.red0 : 0) + (kb + i) * BK;
                            const uint32_t dst = (load_a ? a_base : b_base) + (stage * KPS + i) * (load_a ? A_BYTES : p.b_bytes);
                            if (load_a) {
                                if (MODE == kLinFwd) {
                                    tma_load_3d_pair(dst, &tmA, bar, fa, k, it.g);
                                    tma_load_3d_pair(dst + BOX_BYTES, &tmA, bar, fa2, k, it.g);
                                } else if (MODE == kLinDx) {
                                    tma_load_3d_pair(dst, &tmA, bar, k, fa, it.g);
                                } else {
                                    tma_load_2d_pair(dst, &tmA, bar, fa, k);
                                    tma_load_2d_pair(dst + BOX_BYTES, &tmA, bar, fa2, k);
                                }
                            } else if (B_MN) {
                                tma_load_2d_pair(dst, &tmB, bar, b_row, k);
                                if (nb > 1) tma_load_2d_pair(dst + BOX_BYTES, &tmB, bar, b_row + 64, k);
                            } else {
                                tma_load_2d_pair(dst, &tmB, bar, k, b_row);
                                for (int j = 1; j < nb; ++j)
                                    tma_load_2d_pair(dst + j * b_box, &tmB, bar, k, b_row + j * p.bx);
                            }
                        }
                    }
                    __syncwarp();
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (ADAPT && adapts && ok) {
                    if (!listed) {
                        grid_dependency_wait();
                        listed = true;
                        count = word_now(list_at(it)), id = id_of(it, 0);
                        seen = 1;
                    }
                    if (seen == 1) flags_of(id, flags);
                    adapter_blocks(1 << 30);
                    first_tile = false;
                }
                // (what the next waits are for waits for the kernel before: their limit starts when it has ended)
                if (ADAPT && !load_a) grid_dependency_wait();
            }
            if (!ok) aborted = true;
            __syncwarp();
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issuer (even CTA)
            // (the whole warp walks, one elected lane issues: the descriptors then stay in uniform
            // registers; a loop in one lane took 610 cycles a k-block, more than its MMAs)
            if (rank == 0) {
                Walk<MODE> walk(p, off, cum, pair, npairs);
                Item it;
                int stage = 0, buf = 0;
                uint32_t phase = 0, buf_phase = 0;
                uint32_t tails = 0;  // bit s: parity of stage s's next tail
                bool listed = false;  // ADAPT: the lists are there
                int place = 0;
                uint32_t place_phase = 0;
                bool ok = true;
                // descriptors of stage 0; a stage or a step of 16 along K moves the start address
                constexpr uint32_t A_STEP = A_MN ? UMMA_K * 128 : UMMA_K * 2, B_STEP = B_MN ? UMMA_K * 128 : UMMA_K * 2;
                const uint64_t a_desc0 = smem_desc_sw128(smem_u32(smem_a), A_MN ? BOX_BYTES : 16, 1024);
                const uint64_t b_desc0 = smem_desc_sw128(smem_u32(smem_b), B_MN ? BOX_BYTES : 16, 1024);
                while (ok && walk.next(it)) {
                    const uint32_t idesc = p.idesc | ((uint32_t)(it.w >> 3) << 17);
                    const int kc = CHUNKED ? p.kc : it.kb1 - it.kb0;
                    int count = 0;  // ADAPT: adapters of the tile
                    if (ADAPT && listed && it.kb1 == p.kb) count = word_now(list_at(it));
                    for (int kb0 = it.kb0; kb0 < it.kb1 && ok; kb0 += kc) {
                        if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&tempty_bar[buf]), buf_phase ^ 1, p.limit_ns,
                                                                       abort_flag))) {
                            record_error(p.status, kDevTimeoutMma, abort_flag);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * MAX_W);
                        const int kb1 = min(kb0 + kc, it.kb1);
                        for (int kb = kb0; kb < kb1; kb += KPS) {
                            if (ADAPT && kb == kb0 + p.stages * KPS && !listed && it.kb1 == p.kb) {
                                grid_dependency_wait();
                                listed = true;
                                count = word_now(list_at(it));
                            }
                            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full_bar[stage]), phase, p.limit_ns, abort_flag))) {
                                record_error(p.status, kDevTimeoutMma, abort_flag);
                                ok = false;
                                break;
                            }
                            if (MODE == kLinDw && p.offsets && it.red_rows - kb * BK < BK) {
                                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&peer_bar[stage]), (tails >> stage) & 1,
                                                                               p.limit_ns, abort_flag))) {
                                    record_error(p.status, kDevTimeoutMma, abort_flag);
                                    ok = false;
                                    break;
                                }
                                tails ^= 1u << stage;
                            }
                            tc_fence_after();
                            const bool tail = MODE == kLinDw && p.offsets && it.red_rows - kb * BK < BK;
                            const int steps = tail ? (it.red_rows - kb * BK + UMMA_K - 1) / UMMA_K : BK / UMMA_K;
                            const int n = KPS == 1 ? 1 : min(KPS, kb1 - kb);
                            if (elect_one()) {
#pragma unroll
                                for (int i = 0; i < KPS; ++i) {
                                    if (i >= n) break;
                                    const int at = stage * KPS + i;
                                    const uint64_t a_desc = a_desc0 + (uint32_t)(at * A_BYTES >> 4);
                                    const uint64_t b_desc = b_desc0 + (uint32_t)(at * p.b_bytes >> 4);
#pragma unroll
                                    for (int k = 0; k < BK / UMMA_K; ++k)
                                        if (MODE != kLinDw || k < steps)
                                            umma_f16_pair(d_tmem, a_desc + k * (A_STEP >> 4), b_desc + k * (B_STEP >> 4),
                                                          idesc, (kb + i > kb0 || k > 0) ? 1u : 0u);
                                }
                                umma_commit_mask(smem_u32(&empty_bar[stage]), pair_mask);
                            }
                            __syncwarp();
                            if (++stage == p.stages) {
                                stage = 0;
                                phase ^= 1;
                            }
                        }
                        if constexpr (ADAPT) {
                            if (ok && !listed && it.kb1 == p.kb) {
                                grid_dependency_wait();
                                listed = true;
                                count = word_now(list_at(it));
                            }
                            for (int k = 0; k < count * ad.rs && ok; k += BK) {
                                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&there_bar[place]), place_phase, p.limit_ns,
                                                                               abort_flag))) {
                                    record_error(p.status, kDevTimeoutMma, abort_flag);
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                const int steps = min(BK, count * ad.rs - k) / UMMA_K;  // (the rest of the place is not there)
                                if (elect_one()) {
                                    const int at = p.stages * KPS + place;
                                    const uint64_t a_desc = a_desc0 + (uint32_t)(at * A_BYTES >> 4);
                                    const uint64_t b_desc = b_desc0 + (uint32_t)(at * p.b_bytes >> 4);
#pragma unroll
                                    for (int s = 0; s < BK / UMMA_K; ++s)
                                        if (s < steps)
                                            umma_f16_pair(d_tmem, a_desc + s * (A_STEP >> 4), b_desc + s * (B_STEP >> 4), idesc, 1u);
                                    umma_commit_mask(smem_u32(&free_bar[place]), pair_mask);
                                }
                                __syncwarp();
                                if (++place == ad.places) {
                                    place = 0;
                                    place_phase ^= 1;
                                }
                            }
                        }
                        if (!ok) break;
                        if (elect_one()) umma_commit_mask(smem_u32(&tfull_bar[buf]), pair_mask);
                        __syncwarp();
                        if (++buf == 2) {
                            buf = 0;
                            buf_phase ^= 1;
                        }
                    }
                }
                if (!ok) aborted = true;
                if (elect_one()) umma_commit_mask(smem_u32(drain_bar), pair_mask);
                __syncwarp();
            }
            // (the odd CTA's warp is here from the start)
            if (ADAPT) grid_dependency_wait();
            if (!mbar_wait_while(smem_u32(drain_bar), 0, p.limit_ns, nullptr, progress)) {
                record_error(p.status, kDevTimeoutDrain, abort_flag);
                aborted = true;
            }
            __syncwarp();
        } else if (MODE == kLinDw && warp == 2) {
            // ---------------------------------------------------------------- fixer (both CTAs)
            Walk<MODE> walk(p, off, cum, pair, npairs);
            Item it;
            int stage = 0;
            uint32_t used = 0;  // bit s: parity of stage s's next tail
            bool ok = true;
            while (ok && p.offsets && walk.next(it)) {
                const int nk = it.kb1 - it.kb0;
                if (nk == 0) continue;
                const int r = it.red_rows - (it.kb1 - 1) * BK;  // rows of the last k-block
                const int s = (stage + nk - 1) % p.stages;
                stage = (stage + nk) % p.stages;
                if (r >= BK) continue;
                const uint32_t parity = (used >> s) & 1;
                // (whole tiles go by unseen before it)
                ok = mbar_wait_while(smem_u32(&tail_bar[s]), parity, p.limit_ns, abort_flag, progress);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    if (lane == 0) record_error(p.status, kDevTimeoutMma, abort_flag);
                    aborted = true;
                    break;
                }
                used ^= 1u << s;
                // rows r .. up to the MMA's next multiple of 16, 128 bytes each, in every box
                const int r1 = (r + UMMA_K - 1) / UMMA_K * UMMA_K;
                const int nb = (it.w / 2 + 63) / 64;
                const int chunks = (r1 - r) * 8;
                for (int b = 0; b < 2 + nb; ++b) {
                    uint8_t* box = b < 2 ? smem_a + s * A_BYTES + b * BOX_BYTES
                                         : smem_b + s * p.b_bytes + (b - 2) * BOX_BYTES;
                    for (int c = lane; c < chunks; c += 32)
                        *reinterpret_cast<uint4*>(box + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
                __syncwarp();
                // (the MMA warp waits for both CTAs' fixers, so that they need not for each other)
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(smem_u32(&full_bar[s]));
                    else mbar_arrive_cluster(mapa_shared(smem_u32(&peer_bar[s]), 0));
                }
            }
            __syncwarp();
        } else if (ADAPT && warp == 2) {
            // ---------------------------------------------------------------- the rows' U (both CTAs)
            Walk<MODE> walk(p, off, cum, pair, npairs);
            Item it;
            int place = 0;
            uint32_t place_phase = 0;
            bool ok = true;
            uint16_t* const slots = reinterpret_cast<uint16_t*>(cum + p.G + 1);
            uint8_t* const own_b = smem_b + p.stages * KPS * p.b_bytes;
            grid_dependency_wait();
            while (ok && walk.next(it)) {
                if (it.kb1 != p.kb) continue;
                const int count = word_now(list_at(it)), half = it.w / 2, first = (int)rank * half;
                if (count == 0) continue;
                __syncwarp();
                for (int j = lane; j < half; j += 32)
                    slots[j] = first + j < it.valid && in_range(it.row0 + first + j, p.rows) ? __ldcg(ad.slot + it.row0 + first + j)
                                                                                            : (uint16_t)0xffff;
                __syncwarp();
                const int c = lane % 8;  // a lane has the same eight of K of every fourth row
                int mine = 0;            // lane i: adapter 32 n + i of the list
                // A place whose copies have landed: an unusable adapter's rows, and on to the MMA warp.
                const auto pass_on = [&](int at, int own, bool broken) {
                    if (broken)
                        for (int j = lane / 8; j < half; j += 4)
                            if (slots[j] == own)
                                *reinterpret_cast<uint4*>(own_b + at * p.b_bytes + j * 128 + ((c ^ (j & 7)) << 4)) =
                                    make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&there_bar[at]), 0));
                };
                int last = -1, last_own = 0;  // the place whose copies are under way
                bool last_broken = false;
                for (int k = 0; k < count * ad.rs; k += BK) {
                    const int s0 = k / ad.rs;
                    if (s0 % 32 == 0 && k == s0 * ad.rs) {
                        uint4 flags[2];
                        const int id = id_of(it, s0);
                        flags_of(id, flags);
                        mine = usable(id, flags);
                    }
                    // (a whole tile may go by before the place is free; with one place, what is under way must land first)
                    if (last >= 0 && ad.places == 1) {
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        pass_on(last, last_own, last_broken);
                        last = -1;
                    }
                    ok = __all_sync(0xffffffffu, mbar_wait_while(smem_u32(&free_bar[place]), place_phase ^ 1, p.limit_ns, abort_flag,
                                                                 progress));
                    if (!ok) {
                        if (lane == 0) record_error(p.status, kDevTimeoutProducer, abort_flag);
                        aborted = true;
                        break;
                    }
                    const int own = (k + c * 8) / ad.rs, k0 = k + c * 8 - own * ad.rs;
                    const bool broken = __shfl_sync(0xffffffffu, mine, own % 32) == ad.n && own < count;
                    const uint32_t dst = smem_u32(own_b + place * p.b_bytes);
                    const uint16_t* src = ad.u + (int64_t)(it.row0 + first) * ad.rs + k0;
#pragma unroll 4
                    for (int j = lane / 8; j < half; j += 4) {
                        const bool is = slots[j] == own;
                        copy_async_16(dst + j * 128 + ((c ^ (j & 7)) << 4), is ? src + (int64_t)j * ad.rs : ad.u, is ? 16 : 0);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (last >= 0) {
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        pass_on(last, last_own, last_broken);
                    }
                    last = place, last_own = own, last_broken = broken;
                    if (++place == ad.places) {
                        place = 0;
                        place_phase ^= 1;
                    }
                }
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                if (ok && last >= 0) pass_on(last, last_own, last_broken);
            }
            __syncwarp();
        } else if (MODE == kLinDx && warp == 2) {
            if (p.db) add_db(p, off, lane);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        // ---------------------------------------------------------------- epilogue (both CTAs)
        // ADAPT: bias and residual are read through L1, which is certain to be fresh only behind this; and the limit
        // of the first wait starts when the kernel before has ended.
        if (ADAPT) grid_dependency_wait();
        const int q = warp & 3;             // TMEM lane quarter
        const int group = (warp - EPI_WARP0) / 4;   // takes column blocks group, group + 2, ...
        const int e = threadIdx.x - 32 * EPI_WARP0;
        uint32_t* stg = reinterpret_cast<uint32_t*>(after + (warp - EPI_WARP0) * STG_BYTES);
        int buf = 0;
        uint32_t buf_phase = 0;
        // After a wait has run out a warp goes on through its items without waiting or
        // storing, so that the others' barriers are still met.
        bool dead = false;
        if (p.test_stall < 0 || p.test_stall == pair + 1) {
            bool ok = mbar_wait_cluster(smem_u32(never_bar), 0, p.limit_ns, nullptr);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok && lane == 0) record_error(p.status, kDevTimeoutEpilogue, abort_flag);
            dead = true;
        }
        const int64_t slot_floats = (int64_t)2 * p.ws_cols * CTA_F;  // a slice of the workspace (both CTAs)
        float* const parts = p.ws + (int64_t)rank * p.ws_cols * CTA_F + q * 32 + lane;
        Walk<MODE> walk(p, off, cum, pair, npairs);
        Item it;
        float acc[CHUNKED ? 2 : 1][32];  // one chunk: blocks come straight from tensor memory
        while (walk.next(it)) {
            // columns of a warp's block: up to 32 rows are shared by both groups
            const int bw = it.w <= 16 ? 8 : it.w <= 32 ? 16 : 32, cb0 = group * bw, cb_step = EPI_GROUPS * bw;
            // columns cb .. cb + 31 of the finished accumulator
            const auto fetch_block = [&](int cb, uint32_t(&u)[32]) {
                tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * MAX_W + cb), u);
                tmem_ld_wait();
            };
            const auto wait_full = [&] {
                bool ok = dead ? false : mbar_wait(smem_u32(&tfull_bar[buf]), buf_phase, p.limit_ns, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok && !dead) {
                    if (lane == 0) record_error(p.status, kDevTimeoutEpilogue, abort_flag);
                    dead = true;
                }
                if (ok && warp == EPI_WARP0 && lane == 0) *progress = *progress + 1;
                tc_fence_after();
            };
            const auto release = [&] {
                tc_fence_before();
                __syncwarp();
                // (a cluster-scope release would wait for this tile's stores: 2000 cycles a tile)
                if (lane == 0) mbar_arrive_cluster_light(mapa_shared(smem_u32(&tempty_bar[buf]), 0));
                if (++buf == 2) {
                    buf = 0;
                    buf_phase ^= 1;
                }
            };
            const bool any = it.kb0 < it.kb1;  // (a group without rows: zeros)
            if constexpr (CHUNKED) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[j][i] = 0.f;
                for (int kb0 = it.kb0; kb0 < it.kb1 && !dead; kb0 += p.kc) {
                    wait_full();
                    if (dead) break;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (cb0 + j * cb_step < it.w) {
                            uint32_t u[32];
                            fetch_block(cb0 + j * cb_step, u);
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[j][i] = __fadd_rn(acc[j][i], __uint_as_float(u[i]));
                        }
                    release();
                }
            } else if (any) {
                wait_full();
            }
            if (it.part >= 0) {
                // publish this slice; the CTA that counts last adds the tile's slices in K order
                if (!dead && in_range(walk.slot(), npairs)) {
                    float* mine = parts + walk.slot() * slot_floats;
                    const auto publish = [&](int cb, const float(&v)[32]) {
                        const int n = min(bw, it.w - cb);
                        if (!in_range(cb + n - 1, p.ws_cols)) return;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (i < n)
#pragma unroll
                                for (int k = 0; k < 8; ++k) __stcg(mine + (cb + i + k) * CTA_F, v[i + k]);
                    };
                    if constexpr (CHUNKED) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (cb0 + j * cb_step < it.w) publish(cb0 + j * cb_step, acc[j]);
                    } else {
#pragma unroll 1
                        for (int cb = cb0; cb < it.w; cb += cb_step) {
                            uint32_t u[32];
                            fetch_block(cb, u);
                            float v[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                            publish(cb, v);
                        }
                        release();
                    }
                    __threadfence();
                }
                if (dead) *abort_flag = 1;
                named_barrier(1, 32 * EPI_WARPS);
                if (e == 0) {
                    // A CTA that gave up is counted as well (it comes here all the same), with
                    // SLICE_MISSING: so the count always gets to the last and back to zero, and a tile
                    // that lacks a slice is finished by nobody
                    unsigned* c = p.cnt + 2 * it.part + rank;
                    const unsigned mine = *abort_flag ? 1u + SLICE_MISSING : 1u, now = atomicAdd(c, mine) + mine;
                    int last = now % SLICE_MISSING == (unsigned)walk.slices_of_tile();
                    if (last) {
                        *c = 0;  // ready for the next launch
                        last = now < SLICE_MISSING;
                    }
                    __threadfence();
                    *last_flag = last;
                }
                named_barrier(1, 32 * EPI_WARPS);
                const int last = *last_flag;
                // (read by every warp before the next item's first barrier lets thread 0 on)
                if (!last) continue;
                __threadfence();
            }
            // feature of lane 0, and the column of W it comes from
            const int fw = it.f0 * TILE_F + (GATED ? 64 * (int)rank + 32 * (q & 1) : CTA_F * (int)rank + 32 * q);
            const int nf = dead ? 0 : p.F - fw;
            const int zw = GATED && q >= 2 ? p.F + fw : fw;
            float bias = 0.f;
            if (MODE == kLinFwd && p.bias && lane < nf && in_range(it.g, p.G) && in_range(zw + lane, p.bias_stride))
                bias = from_16<BF16>(static_cast<const uint16_t*>(p.bias)[it.g * p.bias_stride + zw + lane]);
            const int64_t out0 = MODE == kLinDw ? it.g * p.out_stride : 0;
            constexpr int OUT_N = GATED ? 16 : 32;       // rows a warp finishes of 32 (gated: the pair shares them)
            const int own = GATED && q >= 2 ? 16 : 0;    // and the first of them
            const bool residual = MODE == kLinFwd && p.R && !p.out_f32;
            Matrix16 mr = {}, mo = {}, mz = {};
            Ahead<OUT_N> ahead;
            const auto block = [&](const void* base, int64_t ld, int col, int cb, int cb_end, bool vec) {
                const int64_t row = it.row0 + cb;
                const int n = min(it.valid, cb_end) - cb;
                const bool in = n <= 0 || in_range(row + min(n, 32) - 1, p.rows);
                return Matrix16{static_cast<uint16_t*>(const_cast<void*>(base)) + row * ld + col, (int)ld, in ? n : 0, nf, vec};
            };
            const bool fetch = !CHUNKED && any && it.part < 0 && !dead;
            // (chunked: the sums move down a block an iteration, so that one copy of the code does)
#pragma unroll 1
            for (int cb = cb0; cb < it.w; cb += cb_step) {
                float(&v)[32] = acc[0];
                // the residual's loads run while the sums are fetched and activated (a slice's
                // addition needs the registers: after it)
                if (residual) mr = block(p.R, p.ldr, fw, cb + own, cb + bw, p.vec_r);
                if (residual && it.part < 0) ahead.load(mr, lane);
                if (fetch) {
                    uint32_t u[32];
                    fetch_block(cb, u);
                    if (cb + cb_step >= it.w) release();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                } else if (!CHUNKED) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                }
                if (it.part >= 0) {
                    // every slice, this CTA's own included, is read back, COLS columns of DEEP slices
                    // at a time so that their latencies overlap, and added in K order
                    constexpr int DEEP = CHUNKED ? 4 : SUM_DEEP, COLS = 8;
                    const int S = walk.slices_of_tile();
#pragma unroll
                    for (int h = 0; h < 32; h += COLS) {
                        if (h >= bw || cb + h >= it.w) break;
                        for (int c = 0; c < S; c += DEEP) {
                            float t[DEEP][COLS];
#pragma unroll
                            for (int s = 0; s < DEEP; ++s)
                                if (c + s < S) {
                                    const float* src = parts + (it.slot0 + c + s) * slot_floats + (cb + h) * CTA_F;
#pragma unroll
                                    for (int i = 0; i < COLS; ++i) t[s][i] = __ldcg(src + i * CTA_F);
                                }
#pragma unroll
                            for (int s = 0; s < DEEP; ++s)
                                if (c + s < S)
#pragma unroll
                                    for (int i = 0; i < COLS; ++i)
                                        v[h + i] = c + s == 0 ? t[s][i] : __fadd_rn(v[h + i], t[s][i]);
                        }
                    }
                    if (residual) ahead.load(mr, lane);
                }
                if (MODE == kLinFwd) {
                    if (p.bias)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += bias;
                    if (p.Z) {
                        mz = block(p.Z, p.ldz, zw, cb, cb + bw, p.vec_z);
                        store_block<BF16>(mz, stg, lane, v);
                    }
                }
                const auto finish = [&](auto& h) {
                    if (CHUNKED && MODE != kLinDx && p.out_f32) {
                        const int64_t row = it.row0 + cb + own;
                        const int n = min(it.valid, cb + bw) - cb - own;
                        if (n <= 0 || !in_range(row + min(n, OUT_N) - 1, p.rows)) return;
                        store_f32(MODE == kLinFwd && p.R ? static_cast<const float*>(p.R) + row * p.ldr + fw + lane : nullptr,
                                  p.ldr, static_cast<float*>(p.out) + out0 + row * p.ldo + fw + lane, p.ldo, n, lane < nf, h);
                        return;
                    }
                    if (residual) add_block<BF16>(mr, ahead, stg, lane, h);
                    mo = block(static_cast<const uint16_t*>(p.out) + out0, p.ldo, fw, cb + own, cb + bw, p.vec_out);
                    store_block<BF16>(mo, stg, lane, h);
                };
                if constexpr (GATED) {
                    // gate warps finish rows 0..15, up warps 16..31; each leaves the other's part in
                    // its own staging block
                    const bool up = q >= 2;
                    float* mine = reinterpret_cast<float*>(stg) + lane;
                    const float* other = reinterpret_cast<const float*>(
                                             after + (warp - EPI_WARP0 + (up ? -2 : 2)) * STG_BYTES) + lane;
#pragma unroll
                    for (int i = 0; i < 16; ++i) mine[i * 32] = up ? v[i] : v[16 + i];
                    named_barrier(2 + (q & 1) + 2 * group, 64);
                    float h[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float o = other[i * 32];
                        h[i] = up ? silu(o) * v[16 + i] : silu(v[i]) * o;
                    }
                    named_barrier(2 + (q & 1) + 2 * group, 64);
                    finish(h);
                } else {
                    if (MODE == kLinFwd) activate(v, p.act);
                    finish(v);
                }
                if constexpr (CHUNKED) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i];
                }
            }
            // (a warp without a block of its own lets go of the accumulator all the same)
            if (fetch && cb0 >= it.w) release();
        }
        if (dead) aborted = true;
    }

    if (__syncthreads_or(aborted ? 1 : 0)) grace_period(2000000ull);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 2 * MAX_W);
    }
}

template <int MODE, bool GATED, bool BF16, bool CHUNKED, int KPS>
__global__ void __launch_bounds__(THREADS, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, LinParams p)
{
    linear_pair_body<MODE, GATED, BF16, CHUNKED, KPS, false>(tmA, tmB, tmA, p, AdaptParams{});
}

// ------------------------------------------------------------------ host side

// 16-bit tensor [d2][d1][d0] (d0 contiguous) with strides of s1 and s2 elements; 128-byte
// swizzled boxes of 64 x box1.  rank 2 ignores d2.
bool encode(CUtensorMap* map, int rank, const void* base, bool bf16, int64_t d0, int64_t d1, int64_t d2, int64_t s1,
            int64_t s2, int box1)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box1, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct LinPlan {
    int rows, F, kb, f_tiles, wcap, wmax, pairs;
    int bx, b_bytes, kps, stages, places, smem;  // places: beside the ring, for the adapters' blocks
    bool gated, ragged;
    int split_w;  // 0: the last wave is not cut
    int64_t tiles;  // an upper bound when the groups' rows are only known on the device
};

// The tile width for `rows` rows: the multiple of 16 whose tiles take least by the estimates
// above, waves of tiles and a last wave's slices counted (4096 x 4096 outputs: 304 tiles of
// 224 rows are four whole waves of 76 pairs, 256 tiles of 256 rows are 3.4).
int choose_width(int mode, int rows, int f_tiles, int kb, int pairs, int cap, bool split)
{
    if (mode == kLinDw && rows <= 128) return rows < 16 ? 16 : (rows + 15) / 16 * 16;  // one tile
    int best = 16;
    double least = 0;
    const int step = mode == kLinDw ? 128 : 16;
    for (int c = step; c <= cap; c += step) {
        const int w = tile_width(mode, rows, c);
        const int64_t tiles = (int64_t)((rows + w - 1) / w) * f_tiles;
        const int rem = (int)(tiles % pairs);
        const int S = split ? slices(rem, kb, pairs, w) : 1;
        double t = (double)(tiles / pairs) * kb * kb_cycles(w) + 25 * w;  // (and the last epilogue)
        if (rem > 0) t += (double)((kb + S - 1) / S) * kb_cycles(w) + split_cycles(S, w);
        if (c == step || t < least) least = t, best = w;
    }
    return best;
}

LinPlan plan(const LinArgs& a, int num_sms, bool chunked)
{
    LinPlan pl;
    pl.gated = a.mode == kLinFwd && a.act == GEMM_ACT_SWIGLU;
    pl.rows = (int)(a.mode == kLinDw ? a.K : a.M);
    pl.F = (int)(a.mode == kLinFwd ? a.N : a.mode == kLinDx ? a.K : a.Nw);
    const int64_t red = a.mode == kLinFwd ? a.K : a.mode == kLinDx ? a.Nw : a.M;
    pl.kb = (int)((red + BK - 1) / BK);
    const int tile_f = pl.gated ? CTA_F : 2 * CTA_F;
    pl.f_tiles = (pl.F + tile_f - 1) / tile_f;
    const int G = a.G > 0 ? a.G : 1;
    const bool ragged = pl.ragged = a.G > 0 && a.mode != kLinDw;  // the tiles' widths are known on the device only
    // (groups of few rows on average: narrow tiles, which stream the weights faster)
    const int cap = chunked || (ragged && a.M <= 64 * (int64_t)G) ? NARROW_W : MAX_W;
    pl.pairs = num_sms / 2;
    pl.wcap = ragged ? cap
              : a.mode == kLinDw && a.G > 0
                  ? choose_width(a.mode, pl.rows, pl.f_tiles * G, (pl.kb + G - 1) / G, pl.pairs, cap, false)
                    : choose_width(a.mode, pl.rows, pl.f_tiles, pl.kb, pl.pairs, cap, true);
    pl.wmax = ragged ? (int)(a.M < cap ? (a.M + 15) / 16 * 16 : cap) : pl.wcap;
    int64_t row_tiles = (pl.rows + pl.wcap - 1) / pl.wcap;
    if (ragged) row_tiles += a.G < a.M ? a.G : a.M;
    pl.tiles = row_tiles * pl.f_tiles * (a.mode == kLinDw ? G : 1);
    // rows of a TMA box of the K-major B operand: a whole half tile where its height is
    // known, else pieces of a typical group's half tile
    int typical = pl.wmax / 2;
    if (ragged) {
        const int64_t mean = (a.M + a.G - 1) / a.G;
        typical = mean >= 128 ? 64 : mean >= 32 ? 32 : 16;
        if (typical > pl.wmax / 2) typical = pl.wmax / 2;
    }
    pl.bx = typical < 8 ? 8 : (typical + 7) / 8 * 8;
    const int b_rows = (pl.wmax / 2 + pl.bx - 1) / pl.bx * pl.bx;
    pl.b_bytes = a.mode == kLinDw ? (pl.wmax / 2 + 63) / 64 * BOX_BYTES : (b_rows * 128 + 1023) / 1024 * 1024;
    const int fixed = 1024 + EPI_WARPS * STG_BYTES + (4 * MAX_STAGES + 6) * 8 + 16 + 2 * (G + 1) * 4 + 16 +
                      (a.adapt ? ADAPT_SMEM : 0);
    // Narrow tiles: two k-blocks a stage, so that waiting for it and committing it, some 300
    // cycles, take less than its copies and MMAs (per k-block 295 cycles instead of 400 at 16
    // rows, 404 instead of 430 at 160; at 192 it would be 594 instead of 400: three stages).
    // dW's fixer counts stages by k-block.
    pl.kps = a.mode != kLinDw && pl.wmax <= 160 ? 2 : 1;
    pl.places = !a.adapt ? 0 : pl.kps == 1 ? 1 : 4;
    pl.stages = ((SMEM_MAX - fixed) / (A_BYTES + pl.b_bytes) - pl.places) / pl.kps;
    if (pl.stages > MAX_STAGES) pl.stages = MAX_STAGES;
    pl.smem = fixed + (pl.stages * pl.kps + pl.places) * (A_BYTES + pl.b_bytes);
    // groups' dW tiles have lengths of their own and are not cut
    pl.split_w = a.mode == kLinDw && a.G > 0 ? 0 : pl.wmax;
    if (ragged && a.M > a.G) {
        const int64_t mean = (a.M + a.G - 1) / a.G;
        if (mean < pl.wmax) pl.split_w = (int)((mean + 15) / 16 * 16);
    }
    return pl;
}

// One kernel and the clusters of it that can be resident at once (`fit` and `allowed` are the kernel's own:
// cached per process; every device a process drives is taken to be the same part).
template <typename Kernel, typename... Args>
int launch_kernel(Kernel kern, std::atomic<int>& fit, std::atomic<uint64_t>& allowed, const LinPlan& pl, int split_w,
                  int num_sms, cudaStream_t stream, const Args&... args)
{
    if (allow_smem(kern, SMEM_MAX, allowed) != cudaSuccess) return GEMM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_MAX;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // set-up (barriers, tensor memory, descriptors) overlaps the end of the kernel before
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = fit.load();
    if (clusters == 0) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return GEMM_ERR_CUDA;
        if (fa.numRegs < LAUNCH_REGS) return GEMM_ERR_UNSUPPORTED;  // the epilogue would wait for registers
        if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) {
            (void)cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        fit.store(clusters);
    }
    if (clusters > num_sms / 2) clusters = num_sms / 2;
    // pairs with nothing to do are not launched (where the host knows the tiles)
    if (pl.tiles < clusters) {
        if (split_w == 0) clusters = (int)pl.tiles;
        else if (!pl.ragged) clusters = (int)pl.tiles * slices((int)pl.tiles, pl.kb, clusters, split_w);
    }
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.numAttrs = 2;
    cfg.dynamicSmemBytes = pl.smem;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <int MODE, bool GATED, bool BF16, bool CHUNKED, int KPS>
int launch_plain(const LinPlan& pl, const CUtensorMap& tmA, const CUtensorMap& tmB, const LinParams& p, int num_sms,
                 cudaStream_t stream)
{
    static std::atomic<int> fit{0};
    static std::atomic<uint64_t> allowed{0};
    return launch_kernel(linear_pair_kernel<MODE, GATED, BF16, CHUNKED, KPS>, fit, allowed, pl, p.split_w, num_sms, stream,
                         tmA, tmB, p);
}

bool is_chunked(const LinArgs& a, int kc)
{
    const int64_t red = a.mode == kLinFwd ? a.K : a.mode == kLinDx ? a.Nw : a.M;
    return a.out_f32 || kc > 0 || red > (int64_t)MAX_KB_WHOLE * BK;
}

// The kernel's parameters and tensor maps.  Returns a gemm_status_t.
int set_up(const LinArgs& a, const LinPlan& pl, const LinWorkspace& ws, int* dev_status, uint64_t limit_ns, int kc,
           int test_stall, LinParams& p, CUtensorMap& tmA, CUtensorMap& tmB)
{
    if (pl.tiles > 0x7fffffffLL || pl.stages < 2) return GEMM_ERR_UNSUPPORTED;
    p = {};
    p.M = (int)a.M;
    p.rows = pl.rows;
    p.F = pl.F;
    p.kb = pl.kb;
    p.G = a.G > 0 ? a.G : 1;
    p.offsets = a.G > 0 ? a.offsets : nullptr;
    p.f_tiles = pl.f_tiles;
    p.per_inv = (unsigned)((1ull << 32) / (unsigned)(RASTER * pl.f_tiles));
    p.wcap = pl.wcap;
    p.bx = pl.bx;
    p.b_bytes = pl.b_bytes;
    p.stages = pl.stages;
    p.kc = kc > 0 ? (kc + 1) / 2 * 2 : 16;  // (chunks end on whole stages)
    p.split_w = ws.partials && ws.counters ? pl.split_w : 0;
    p.bias = a.bias;
    p.bias_stride = a.Nw;
    p.R = a.R;
    p.ldr = a.ldr;
    p.Z = a.Z;
    p.ldz = a.ldz;
    p.out = a.out;
    p.ldo = a.ldo;
    p.out_stride = a.out_stride;
    const auto vec = [](const void* q, int64_t ld) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld % 8 == 0; };
    p.vec_r = vec(a.R, a.ldr);
    p.vec_z = vec(a.Z, a.ldz);
    p.vec_out = vec(a.out, a.ldo) && a.out_stride % 8 == 0;
    p.act = a.act;
    p.out_f32 = a.out_f32 ? 1 : 0;
    p.ws = ws.partials;
    p.cnt = ws.counters;
    p.ws_cols = pl.wmax;
    p.status = dev_status;
    p.limit_ns = limit_ns;
    p.test_stall = test_stall;
    p.db = a.db;
    p.db_ws = a.db_ws;
    p.db_piece = a.db_piece;
    p.db_cols = (int)a.Nw;
    const bool a_mn = a.mode != kLinDx, b_mn = a.mode == kLinDw;
    // kind::f16: fp32 accumulator, both operands of one type, MN-major bits, M = 256
    p.idesc = (1u << 4) | ((a.bf16 ? 1u : 0u) << 7) | ((a.bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
              ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(2 * CTA_F >> 4) << 24);
    tmA = {}, tmB = {};
    if (pl.kb > 0) {
        bool ok;
        if (a.mode == kLinDw)
            ok = encode(&tmA, 2, a.dZ, a.bf16, a.Nw, a.M, 1, a.lddz, 0, 64) &&
                 encode(&tmB, 2, a.X, a.bf16, a.K, a.M, 1, a.ldx, 0, 64);
        else
            ok = encode(&tmA, 3, a.W, a.bf16, a.Nw, a.K, p.G, a.ldw, p.G > 1 ? a.w_stride : a.K * a.ldw,
                        a.mode == kLinFwd ? 64 : CTA_F) &&
                 (a.mode == kLinFwd ? encode(&tmB, 2, a.X, a.bf16, a.K, a.M, 1, a.ldx, 0, pl.bx)
                                    : encode(&tmB, 2, a.dZ, a.bf16, a.Nw, a.M, 1, a.lddz, 0, pl.bx));
        if (!ok) return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}
}  // namespace

}  // namespace gemm_gb300
