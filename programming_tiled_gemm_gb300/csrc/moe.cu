// The kernels around the grouped products of a mixture-of-experts block: the router (top-k
// of a softmax over the experts, with the rows sorted by expert), its gradient, and the
// exchange of rows with the experts.
//
// Router: w[t][j] = p[t][e_j] (renormalised: over the k picked), p = softmax(l[t]).  A warp
// takes a token with its logits in registers and picks k times: the largest order-preserving
// 32-bit key over the warp (redux.sync), then the lowest index that has it.  A logit of -inf
// is an expert that is not there: it is never picked.  The rows are then sorted by expert,
// stably: each warp counts its own picks per expert in order, the block adds its
// warps' counts, and the block that counts last adds the blocks' counts; a second kernel
// writes the places.  One block (up to 128 tokens, 64 above 256 experts) does all of it in one launch.  Bound by
// latency and by the picks' integer instructions, not by its few MB: 16 tokens to 4 of 64
// experts 5.3 us, 16384 to 8 of 128 21 us (11 us of it the picks, 7 us the last block's sums)
// and 4 us for the places.
//
// Exchange: bound by memory; 16 bytes a thread, a block a row (dispatch) or a token
// (combine), the sums in fp32 in the order of j.
//
// All but the router's first kernel are launched as dependents of the kernel before them, whose
// results they wait for: 16 tokens' dispatch and combine 3.2 us instead of 3.6.  (That one, a
// dependent of the router's product, made a block of 4096 tokens 2 % slower: 225 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "linear.h"
#include "moe.h"
#include "ptx.h"

namespace gemm_gb300 {

GEMM_DEBUG_UNIT(moe)

namespace {

struct F32 {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
};
struct BF16 {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(__ushort_as_bfloat16(v)); }
    static __device__ __forceinline__ T put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
struct F16 {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ T put(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

// ------------------------------------------------------------------ router

constexpr int R_EACH = 4;  // tokens of a warp at most
// Warps of a block for C logits a lane (by the registers they take).
__host__ __device__ constexpr int route_warps(int C) { return C <= 8 ? 32 : 16; }

struct RouteParams {
    const void* logits;
    int64_t ld;
    int T, E, k, renorm, nblk;
    int tokens;  // of a block
    float* weights;
    int* experts;
    int* slots;
    int* rows;
    int* offsets;
    int* base;  // [nblk][E]: counts, then each block's first place per expert
    unsigned* cnt;
};

// Larger values have larger keys; NaN (as the largest) before +inf, 0 for -inf.  +0 = -0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// The value of a key (a NaN for any NaN's).
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// C logits a lane: expert 32 c + lane
template <typename D, int C>
__global__ void __launch_bounds__(32 * route_warps(C)) route_kernel(RouteParams p)
{
    constexpr int R_WARPS = route_warps(C), R_THREADS = 32 * R_WARPS;
    // [R_WARPS][E]: a warp's picks per expert, then the places its first picks take in the block
    extern __shared__ uint16_t wc[];
    int* own_counts = reinterpret_cast<int*>(wc + R_WARPS * p.E);  // [E]: a single block's counts, then first places
    __shared__ int last, scan[R_WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int E = p.E, k = p.k;
    const bool one = p.nblk == 1;
    for (int i = threadIdx.x; i < R_WARPS * E; i += R_THREADS) wc[i] = 0;
    __syncthreads();
    // (a single block spreads its tokens over all its warps)
    const int per = one ? (p.T + R_WARPS - 1) / R_WARPS : p.tokens / R_WARPS;
    const int t0 = min(blockIdx.x * p.tokens + warp * per, p.T), n_own = min(per, p.T - t0);
    uint16_t* mine = wc + warp * E;
    const auto fetch = [&](int t, float(&v)[C]) {
        const typename D::T* l = static_cast<const typename D::T*>(p.logits) + (int64_t)t * p.ld;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = 32 * c + lane;
            v[c] = e < E && in_range(t, p.T) ? D::get(l[e]) : -INFINITY;
        }
    };
    int picks[R_EACH], ranks[R_EACH];  // lane j: the j-th pick of each token
    float next[C];
    if (n_own > 0) fetch(t0, next);
#pragma unroll
    for (int q = 0; q < R_EACH; ++q) {
        if (q >= n_own) break;
        const int t = t0 + q;
        float v[C];
        uint32_t key[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            v[c] = next[c];
            key[c] = order_key(v[c]);
        }
        if (q + 1 < n_own) fetch(t + 1, next);  // travels while this token is sorted out
        int pick = -1;
        float val = 0.f, top = 0.f;
        if constexpr (C <= 8) {
            // each lane sorts its keys once (equal ones stay in order); a round then looks at
            // the lanes' heads only: half the instructions of searching all keys again
            uint32_t order = 0x76543210u;  // the keys' c, a nibble each
#pragma unroll
            for (int i = C - 1; i > 0; --i)
#pragma unroll
                for (int c = 0; c < i; ++c) {
                    const bool swap = key[c + 1] > key[c];
                    const uint32_t lo = key[c], hi = key[c + 1];
                    key[c] = swap ? hi : lo;
                    key[c + 1] = swap ? lo : hi;
                    const uint32_t d = ((order >> (4 * c)) ^ (order >> (4 * c + 4))) & 15u;
                    order ^= swap ? (d << (4 * c)) | (d << (4 * c + 4)) : 0u;
                }
            for (int j = 0; j < k; ++j) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
                if (m == 0) break;  // no expert is left
                const uint32_t who = __ballot_sync(0xffffffffu, key[0] == m);
                const int own = (int)(order & 15u) * 32 + lane;
                const int e = (who & (who - 1)) ? (int)__reduce_min_sync(0xffffffffu, key[0] == m ? (unsigned)own : 0xffffffffu)
                                                : __shfl_sync(0xffffffffu, own, __ffs(who) - 1);
                if (own == e) {
#pragma unroll
                    for (int c = 0; c + 1 < C; ++c) key[c] = key[c + 1];
                    key[C - 1] = 0;
                    order >>= 4;
                }
                const float x = key_value(m);
                if (j == 0) top = x;
                if (lane == j) pick = e, val = x;
            }
        } else {
            for (int j = 0; j < k; ++j) {
                uint32_t best = 0;
                int at = 0;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (key[c] > best) best = key[c], at = c;
                const uint32_t m = __reduce_max_sync(0xffffffffu, best);
                if (m == 0) break;
                const int e = (int)__reduce_min_sync(0xffffffffu, best == m ? (unsigned)(32 * at + lane) : 0xffffffffu);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (32 * c + lane == e) key[c] = 0;
                const float x = key_value(m);
                if (j == 0) top = x;
                if (lane == j) pick = e, val = x;
            }
        }
        const bool have = pick >= 0;
        const float ex = have ? expf(val - top) : 0.f;
        float rest = 0.f;
        if (p.renorm) {
            rest = ex;
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (v[c] != -INFINITY) rest += expf(v[c] - top);
        }
        rest = warp_sum(rest);
        // rank among the warp's earlier picks of the same expert (a token's picks differ)
        ranks[q] = have ? mine[pick]++ : 0;
        picks[q] = pick;
        __syncwarp();
        if (lane < k && in_range(t, p.T)) {
            const int64_t i = (int64_t)t * k + lane;
            p.weights[i] = have ? ex / rest : 0.f;
            p.experts[i] = pick;
        }
    }
    __syncthreads();
    // a block's count per expert, and each warp's first place in it
    int* counts = one ? own_counts : p.base + (int64_t)blockIdx.x * E;
    for (int e = threadIdx.x; e < E; e += R_THREADS) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) {
            const int n = wc[w * E + e];
            wc[w * E + e] = (uint16_t)s;
            s += n;
        }
        counts[e] = s;
    }
    __syncthreads();
    // the last block: each block's first place per expert
    if (!one) {
#pragma unroll
        for (int q = 0; q < R_EACH; ++q)
            if (q < n_own && lane < k)
                p.slots[(int64_t)(t0 + q) * k + lane] = picks[q] >= 0 ? ranks[q] + mine[picks[q]] : 0;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            last = atomicAdd(p.cnt, 1u) == (unsigned)(p.nblk - 1);
            if (last) *p.cnt = 0;  // ready for the next launch
            __threadfence();
        }
        __syncthreads();
        if (!last) return;
        __threadfence();
    }
    // chunks of `width` experts, neighbours in neighbouring threads; R_THREADS / width threads
    // an expert, each a stretch of the blocks
    __shared__ int sums[R_THREADS];
    int width = 32;
    while (width < E && width < R_THREADS) width *= 2;
    const int S = R_THREADS / width, part = threadIdx.x / width, col = threadIdx.x % width;
    const int b0 = (int)((unsigned)p.nblk * part / S), b1 = (int)((unsigned)p.nblk * (part + 1) / S);
    int before = 0;  // rows of the earlier chunks' experts
    for (int e0 = 0; e0 < E; e0 += width) {
        const int e = e0 + col;
        int n = 0;
        if (e < E && one) {
            if (part == 0) n = own_counts[e];
        } else if (e < E) {
#pragma unroll 16
            for (int b = b0; b < b1; ++b) n += __ldcg(p.base + (int64_t)b * E + e);
        }
        sums[threadIdx.x] = n;
        __syncthreads();
        // the stretches' sums before each, and the experts' totals
        int total = 0;
        if (part == 0)
            for (int q = 0; q < S; ++q) {
                const int t = sums[q * width + col];
                sums[q * width + col] = total;
                total += t;
            }
        // exclusive scan of the totals
        int s = total;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) scan[warp] = s;
        __syncthreads();
        int low = 0, all = 0;
#pragma unroll
        for (int w = 0; w < R_WARPS; ++w) {
            if (w < warp) low += scan[w];
            all += scan[w];
        }
        if (part == 0) {
            const int first = before + low + s - total;
            if (e < E) p.offsets[e] = first;
            for (int q = 0; q < S; ++q) sums[q * width + col] += first;
        }
        __syncthreads();
        int at = sums[threadIdx.x];
        if (e < E && one) {
            if (part == 0) own_counts[e] = at;
        } else if (e < E) {
            for (int b = b0; b < b1; b += 16) {
                // (sixteen loads before their stores: one latency)
                int m[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) m[i] = b + i < b1 ? __ldcg(p.base + (int64_t)(b + i) * E + e) : 0;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (b + i < b1) {
                        p.base[(int64_t)(b + i) * E + e] = at;
                        at += m[i];
                    }
            }
        }
        before += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) p.offsets[E] = before;
    if (!one) return;
    // (nothing of a single block's places goes through memory: that took 1.1 us of its 6.5)
#pragma unroll
    for (int q = 0; q < R_EACH; ++q)
        if (q < n_own && lane < k) {
            const int i = (t0 + q) * k + lane;
            int slot = -1;
            if (picks[q] >= 0) {
                slot = own_counts[picks[q]] + mine[picks[q]] + ranks[q];
                if (in_range(slot, (int64_t)p.T * k)) p.rows[slot] = i;
            }
            p.slots[i] = slot;
        }
    for (int i = before + (int)threadIdx.x; i < p.T * k; i += R_THREADS) p.rows[i] = -1;
}

__global__ void route_place_kernel(RouteParams p)
{
    grid_dependency_wait();
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, n = (int64_t)p.T * p.k;
    if (i >= n) return;
    const int e = p.experts[i];
    int slot = -1;
    if (e >= 0 && in_range(e, p.E) && in_range(i / p.k / p.tokens, p.nblk)) {
        slot = p.base[(i / p.k / p.tokens) * p.E + e] + p.slots[i];
        if (in_range(slot, n)) p.rows[slot] = (int)i;
    }
    p.slots[i] = slot;
    if (i >= p.offsets[p.E]) p.rows[i] = -1;
}

struct RouteGradParams {
    const float* dweights;
    const void* logits;
    int64_t ld;
    const int* experts;
    int T, E, k, renorm;
    void* dlogits;
    int64_t ldd;
};

constexpr int G_WARPS = 8;

// dl = p (g - sum p g), g the picks' dw (0 elsewhere), p over the picks or over all experts
template <typename D>
__global__ void __launch_bounds__(32 * G_WARPS) route_grad_kernel(RouteGradParams p)
{
    extern __shared__ float up[];  // [G_WARPS][E]
    grid_dependency_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t t = (int64_t)blockIdx.x * G_WARPS + warp;
    if (t >= p.T) return;
    float* g = up + warp * p.E;
    const typename D::T* l = static_cast<const typename D::T*>(p.logits) + t * p.ld;
    typename D::T* o = static_cast<typename D::T*>(p.dlogits) + t * p.ldd;
    for (int e = lane; e < p.E; e += 32) g[e] = 0.f;
    __syncwarp();
    int e = lane < p.k ? p.experts[t * p.k + lane] : -1;
    if (e >= 0 && (!in_range(e, p.E) || e >= p.E)) e = -1;
    const bool have = e >= 0;
    const float dw = have ? p.dweights[t * p.k + lane] : 0.f;
    const float x = have ? D::get(l[e]) : -INFINITY;
    float top = x;  // (a NaN logit makes every gradient NaN through the sums)
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const unsigned any = __ballot_sync(0xffffffffu, have);
    if (p.renorm) {
        const float ex = have ? expf(x - top) : 0.f;
        const float w = ex / warp_sum(ex);
        const float mean = warp_sum(have ? w * dw : 0.f);
        if (have) g[e] = w * (dw - mean);
        __syncwarp();
        for (int i = lane; i < p.E; i += 32) o[i] = D::put(g[i]);
        return;
    }
    float total = 0.f;
    if (any)
        for (int i = lane; i < p.E; i += 32) {
            const float v = D::get(l[i]);
            if (v != -INFINITY) total += expf(v - top);
        }
    total = warp_sum(total);
    const float mean = warp_sum(have ? expf(x - top) / total * dw : 0.f);
    if (have) g[e] = dw;
    __syncwarp();
    for (int i = lane; i < p.E; i += 32) {
        const float v = D::get(l[i]);
        o[i] = D::put(any && v != -INFINITY ? expf(v - top) / total * (g[i] - mean) : 0.f);
    }
}

// ------------------------------------------------------------------ exchange

// V values at p + i (i a multiple of V): one access of up to 16 bytes, or one value
template <typename D, int V>
struct Vec {
    alignas(16) typename D::T v[V];
    __device__ __forceinline__ void load(const void* base, int64_t i)
    {
        const typename D::T* q = static_cast<const typename D::T*>(base) + i;
        if constexpr (V * sizeof(v[0]) == 16) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(q);
        else v[0] = *q;
    }
    __device__ __forceinline__ void store(void* base, int64_t i) const
    {
        typename D::T* q = static_cast<typename D::T*>(base) + i;
        if constexpr (V * sizeof(v[0]) == 16) *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(v);
        else *q = v[0];
    }
    // written once, not read soon: out of L2 first
    __device__ __forceinline__ void store_once(void* base, int64_t i) const
    {
        typename D::T* q = static_cast<typename D::T*>(base) + i;
        if constexpr (V * sizeof(v[0]) == 16) __stcs(reinterpret_cast<uint4*>(q), *reinterpret_cast<const uint4*>(v));
        else *q = v[0];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = D::put(0.f);
    }
};

// xr[r] = x[rows[r] / k], zeros where rows[r] < 0
template <typename D, int V>
__global__ void dispatch_kernel(DispatchArgs a)
{
    grid_dependency_wait();
    const int64_t r = blockIdx.x;
    const int at = a.rows[r];
    const int64_t t = at >= 0 ? at / a.k : -1;
    if (at >= 0 && (!in_range(t, a.T) || t >= a.T)) return;  // (no row of x)
    // four accesses in flight a thread; x's row is read again for the token's other experts,
    // the copies are not.  (8192 x 4096 bf16 to four experts: 59 us, 5.7 TB/s; x comes from DRAM
    // 2.1 times, each die's L2 fetching it once, whatever the order of the rows.)
    const int step = blockDim.x * V;
    for (int c = threadIdx.x * V; c < a.N; c += 4 * step) {
        Vec<D, V> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i * step < a.N && in_range(c + i * step + V - 1, a.N)) {
                if (t >= 0) v[i].load(a.x, t * a.ldx + c + i * step);
                else v[i].zero();
            }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i * step < a.N && in_range(c + i * step + V - 1, a.N)) v[i].store_once(a.xr, r * a.ldxr + c + i * step);
    }
}

constexpr int MAX_K = 32;

// out[t] = sum_j w[t][j] y[slots[t][j]] + R[t] (w = 1 where not given).  8192 x 4096 bf16
// from four experts: 53 us, 6.3 TB/s of rows in and out.
template <typename D, int V>
__global__ void combine_kernel(CombineArgs a)
{
    __shared__ int slot[MAX_K];
    __shared__ float w[MAX_K];
    grid_dependency_wait();
    const int64_t t = blockIdx.x;
    if (threadIdx.x < a.k) {
        const int s = a.slots[t * a.k + threadIdx.x];
        slot[threadIdx.x] = s >= 0 && in_range(s, a.rows_y) && s < a.rows_y ? s : -1;
        w[threadIdx.x] = a.weights ? a.weights[t * a.k + threadIdx.x] : 1.f;
    }
    __syncthreads();
    for (int c = threadIdx.x * V; c < a.N; c += blockDim.x * V) {
        if (!in_range(c + V - 1, a.N)) break;
        float s[V] = {};
        int j = 0;
        // four rows in flight, added in order
        for (; j + 4 <= a.k; j += 4) {
            Vec<D, V> y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (slot[j + i] >= 0) y[i].load(a.y, (int64_t)slot[j + i] * a.ldy + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (slot[j + i] >= 0)
#pragma unroll
                    for (int q = 0; q < V; ++q) s[q] = fmaf(w[j + i], D::get(y[i].v[q]), s[q]);
        }
        for (; j < a.k; ++j)
            if (slot[j] >= 0) {
                Vec<D, V> y;
                y.load(a.y, (int64_t)slot[j] * a.ldy + c);
#pragma unroll
                for (int q = 0; q < V; ++q) s[q] = fmaf(w[j], D::get(y.v[q]), s[q]);
            }
        Vec<D, V> o;
        if (a.R) {
            o.load(a.R, t * a.ldr + c);
#pragma unroll
            for (int q = 0; q < V; ++q) s[q] += D::get(o.v[q]);
        }
#pragma unroll
        for (int q = 0; q < V; ++q) o.v[q] = D::put(s[q]);
        o.store(a.out, t * a.ldo + c);
    }
}

// dy[slots[t][j]] = w[t][j] dout[t], dw[t][j] = <dout[t], y[slots[t][j]]>; dy's rows that
// hold nothing (rows[r] < 0) are zero.  One pass: dout's row stays in L1 for its k uses.
// 8192 x 4096 bf16, four experts: 90 us, 6.7 TB/s.
template <typename D, int V>
__global__ void combine_grad_kernel(CombineGradArgs a)
{
    __shared__ float part[MAX_K][8];
    grid_dependency_wait();
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    for (int j = 0; j < a.k; ++j) {
        const int64_t i = t * a.k + j;
        int s = a.slots[i];
        if (s >= 0 && (!in_range(s, a.T * a.k) || s >= a.T * a.k)) s = -1;
        const float w = a.weights[i];
        float dot = 0.f;
        const bool none = a.rows[i] < 0;  // row i of dy (not of this token) holds nothing
        if (!none) (void)in_range(a.rows[i], a.T * a.k);
        for (int c = threadIdx.x * V; c < a.N; c += blockDim.x * V) {
            if (!in_range(c + V - 1, a.N)) break;
            Vec<D, V> g, y;
            if (s >= 0) {
                g.load(a.dout, t * a.lddo + c);
                y.load(a.y, (int64_t)s * a.ldy + c);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float d = D::get(g.v[q]);
                    dot = fmaf(d, D::get(y.v[q]), dot);
                    g.v[q] = D::put(w * d);
                }
                g.store(a.dy, (int64_t)s * a.lddy + c);
            }
            if (none) {
                y.zero();
                y.store(a.dy, i * a.lddy + c);
            }
        }
        dot = warp_sum(dot);
        if (lane == 0) part[j][warp] = dot;
    }
    __syncthreads();
    if (threadIdx.x < a.k) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += part[threadIdx.x][w];
        a.dweights[t * a.k + threadIdx.x] = s;
    }
}

int row_threads(int64_t N, int V, int each = 1)
{
    const int64_t n = (N + (int64_t)V * each - 1) / ((int64_t)V * each);
    return n >= 256 ? 256 : (int)((n + 31) / 32 * 32);
}

bool aligned(const void* p, int64_t ld, int es) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * es % 16 == 0; }

template <typename D, int C>
cudaError_t launch_route_c(const RouteParams& p, cudaStream_t s)
{
    const size_t smem = route_warps(C) * p.E * sizeof(uint16_t) + (p.nblk == 1 ? p.E * sizeof(int) : 0);
    route_kernel<D, C><<<p.nblk, 32 * route_warps(C), smem, s>>>(p);
    return cudaGetLastError();
}

template <typename D>
cudaError_t launch_route_t(const RouteParams& p, cudaStream_t s)
{
    if (p.E <= 32) return launch_route_c<D, 1>(p, s);
    if (p.E <= 64) return launch_route_c<D, 2>(p, s);
    if (p.E <= 128) return launch_route_c<D, 4>(p, s);
    if (p.E <= 256) return launch_route_c<D, 8>(p, s);
    if (p.E <= 512) return launch_route_c<D, 16>(p, s);
    return launch_route_c<D, 32>(p, s);
}

template <typename F>
cudaError_t by_type(int dtype, F f)
{
    if (dtype == GEMM_F32) return f(F32());
    if (dtype == GEMM_BF16) return f(BF16());
    return f(F16());
}

}  // namespace

namespace {
// Up to four tokens a warp one block does it all; else a warp takes as few tokens as fill the SMs (4096 x
// 256 to eight: 128 blocks of a token a warp 20 us, 32 blocks of four 31 us).
int block_tokens(int64_t T, int64_t E, int num_sms)
{
    const int warps = route_warps(E <= 256 ? 8 : 16);
    if (T <= warps * R_EACH) return warps * R_EACH;
    const int64_t each = (T + (int64_t)num_sms * warps - 1) / ((int64_t)num_sms * warps);
    return warps * (int)(each < R_EACH ? each : R_EACH);
}
}  // namespace

size_t moe_route_ws_bytes(const RouteArgs& a, int num_sms)
{
    const int n = block_tokens(a.T, a.E, num_sms);
    return (size_t)((a.T + n - 1) / n) * a.E * sizeof(int);
}

int launch_moe_route(const RouteArgs& a, int* ws, unsigned* counter, int num_sms, cudaStream_t s, int* launches)
{
    RouteParams p = {};
    p.logits = a.logits;
    p.ld = a.ld;
    p.T = (int)a.T;
    p.E = (int)a.E;
    p.k = a.k;
    p.renorm = a.renormalize;
    p.tokens = block_tokens(a.T, a.E, num_sms);
    p.nblk = (int)((a.T + p.tokens - 1) / p.tokens);
    p.weights = a.weights;
    p.experts = a.experts;
    p.slots = a.slots;
    p.rows = a.rows;
    p.offsets = a.offsets;
    p.base = ws;
    p.cnt = counter;
    const cudaError_t e = by_type(a.dtype, [&](auto d) { return launch_route_t<decltype(d)>(p, s); });
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    if (p.nblk > 1) {
        const int64_t n = a.T * a.k;
        if (launch_dependent(route_place_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p) != cudaSuccess)
            return GEMM_ERR_CUDA;
        *launches += 1;
    }
    return GEMM_OK;
}

int launch_moe_route_grad(const RouteGradArgs& a, cudaStream_t s, int* launches)
{
    RouteGradParams p = {a.dweights, a.logits, a.ld, a.experts, (int)a.T, (int)a.E, a.k, a.renormalize, a.dlogits, a.ldd};
    const cudaError_t e = by_type(a.dtype, [&](auto d) {
        return launch_dependent(route_grad_kernel<decltype(d)>, dim3((unsigned)((a.T + G_WARPS - 1) / G_WARPS)),
                                dim3(32 * G_WARPS), G_WARPS * a.E * sizeof(float), s, p);
    });
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

namespace {

// Rows of 16-byte accesses where every operand allows them, else one value at a time.
template <template <typename, int> class Launch, typename Args>
int launch_rows(const Args& a, int dtype, bool vec, int64_t blocks, cudaStream_t s, int* launches)
{
    if (blocks == 0 || a.N == 0) return GEMM_OK;
    const cudaError_t e = by_type(dtype, [&](auto d) {
        using D = decltype(d);
        constexpr int V = 16 / sizeof(typename D::T);
        if (vec) return Launch<D, V>::run(a, (unsigned)blocks, row_threads(a.N, V, Launch<D, V>::EACH), s);
        return Launch<D, 1>::run(a, (unsigned)blocks, row_threads(a.N, 1, Launch<D, 1>::EACH), s);
    });
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

template <typename D, int V>
struct Dispatch {
    static constexpr int EACH = 4;  // accesses a thread has in flight
    static cudaError_t run(const DispatchArgs& a, unsigned b, int t, cudaStream_t s)
    {
        return launch_dependent(dispatch_kernel<D, V>, dim3(b), dim3(t), 0, s, a);
    }
};
template <typename D, int V>
struct Combine {
    static constexpr int EACH = 1;
    static cudaError_t run(const CombineArgs& a, unsigned b, int t, cudaStream_t s)
    {
        return launch_dependent(combine_kernel<D, V>, dim3(b), dim3(t), 0, s, a);
    }
};
template <typename D, int V>
struct CombineGrad {
    static constexpr int EACH = 1;
    static cudaError_t run(const CombineGradArgs& a, unsigned b, int t, cudaStream_t s)
    {
        return launch_dependent(combine_grad_kernel<D, V>, dim3(b), dim3(t), 0, s, a);
    }
};

}  // namespace

int launch_moe_dispatch(const DispatchArgs& a, int dtype, cudaStream_t s, int* launches)
{
    const int es = dtype == GEMM_F32 ? 4 : 2;
    const bool vec = a.N * es % 16 == 0 && aligned(a.x, a.ldx, es) && aligned(a.xr, a.ldxr, es);
    return launch_rows<Dispatch>(a, dtype, vec, a.T * a.k, s, launches);
}

int launch_moe_combine(const CombineArgs& a, int dtype, cudaStream_t s, int* launches)
{
    const int es = dtype == GEMM_F32 ? 4 : 2;
    const bool vec = a.N * es % 16 == 0 && aligned(a.y, a.ldy, es) && aligned(a.out, a.ldo, es) &&
                     (!a.R || aligned(a.R, a.ldr, es));
    return launch_rows<Combine>(a, dtype, vec, a.T, s, launches);
}

int launch_moe_combine_grad(const CombineGradArgs& a, int dtype, cudaStream_t s, int* launches)
{
    const int es = dtype == GEMM_F32 ? 4 : 2;
    const bool vec = a.N * es % 16 == 0 && aligned(a.y, a.ldy, es) && aligned(a.dout, a.lddo, es) &&
                     aligned(a.dy, a.lddy, es);
    return launch_rows<CombineGrad>(a, dtype, vec, a.T, s, launches);
}

}  // namespace gemm_gb300
