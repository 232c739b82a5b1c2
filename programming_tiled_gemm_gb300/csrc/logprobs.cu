// Log probabilities of given tokens, the entropy and the best alternatives of rows of logits,
// and the logits' gradient.
//
// With c = 1 / (T ln 2) and the row's largest logit m: t_j = (z_j - m) c, S = sum 2^t_j, Q = sum 2^t_j t_j,
//     ln p_j = (z_j - m) / T - ln S,   H = ln S - ln 2 Q / S.
// The difference comes first: t is 0 at the largest logit and below 0 elsewhere, whatever their magnitude, so no
// power overflows and S is 1 at least.  (z c less a rounded m c is one operation instead of two; but from |m| c = 2^31 on
// what m c lost in rounding is beyond 2^t's range, and a masked value of -1e10 reaches that.)  With h = 1/2 it is
// t = (z h - m h) (c / h), as the difference of two finite logits may be beyond fp32's range while t is not.  From c = 2
// on such a t is below -2^128, so that h = 1 will do (and c / h stays finite).
// One pass: every thread keeps its own m, S and Q and rescales them when m grows,
//     S' = f S,  Q' = f (Q + d S),  d = (m - m') c,  f = 2^d,
// and the threads' sums are joined the same way.  As a factor, t is clamped at -1e4, far below
// where 2^t is 0: 0 * -inf is 0 there.
//
// Alternatives: the pass leaves the maxima of units: 64 bytes (four lanes) of a row of the block's vectors, in one or
// more of its batches, so that there are 32 to 256 units a CTA.  The `top` best logits of a CTA's part all belong to
// units whose maximum is among the `top` largest, and none of them is below the smallest of these.  So only those
// units are read again; the few logits that are no worse than that bound wait in shared memory until a warp has 32,
// which it sorts and merges with its best in 6 exchanges of 64-bit keys of logit and index.
//
// A cluster of up to 8 CTAs shares a row where there are few (their sums and lists go to the
// first CTA's shared memory); rows are read with 16-byte loads from the first 16-byte boundary
// on, wherever they start.  One launch each, no workspace, sums in a fixed order.
//
// Bound by memory where the rows fill the SMs, next by the exponentials (16 a cycle and SM: two thirds of the
// reading's time at 16 bits); short calls by latency.  Measured (GPU time; bf16 where not said otherwise):
//   4096 x 131072: forward 157 us, 6.8 TB/s (with entropy 163); with 20 alternatives 228; the gradient 304, 7.1 TB/s
//   1000 x 50257 with entropy: 26 us, 3.9 TB/s (one wave of CTAs, 12 batches a thread); its gradient 33, 6.1 TB/s (31
//   behind the forward pass, which leaves a part of the logits in L2); into rows of another alignment 119
//   64 x 131072 with entropy: 7.7 us; with 20 alternatives 15.0; 1 x 32000 fp32 with entropy and 5 alternatives: 7.8
// z c - R, R the rounded m c, instead of the difference: 4096 x 131072 160 us, with entropy 162, 1000 x 50257 25.2.
// Dropped: every logit offered to sorted lists as the row goes by (64 x 131072, 20 alternatives: 51 us); one maximum a
// thread as the unit (its 16 bytes cost whole sectors again: 4096 x 131072 286 us); units ranked by counting (241, and
// 144 instead of 109 for the best of 4096 x 32000 fp32); persistent blocks for the gradient (552 instead of 494 both
// ways); logits through a ring of asynchronous copies two to four batches ahead instead of one in registers (1000 x
// 50257: 27.5 to 29.3 instead of 27.1); sums two at a time (f32x2) take 161 us where single ones took 169.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "logprobs.h"
#include "ptx.h"

namespace gemm_gb300 {

namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int MAX_CLUSTER = 8;
constexpr int FLY = 4;  // 16-byte loads of a thread in a batch
constexpr int MAX_UNITS = 256;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float FLOOR = -1e4f;  // of exponents: exp2 is 0 there

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Larger values have larger keys; 0 for -inf.  (NaN is not asked for.)  +0 = -0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (v == -INFINITY) return 0u;
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return k == 0 ? -INFINITY : __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct LF32 {
    using T = float;
    static constexpr int PER = 4;  // of 16 bytes
    static constexpr uint32_t LOW = 0xff800000u;  // a word of -inf
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&z)[PER])
    {
        z[0] = __uint_as_float(v.x), z[1] = __uint_as_float(v.y);
        z[2] = __uint_as_float(v.z), z[3] = __uint_as_float(v.w);
    }
    // the largest of FLY vectors (NaN left out)
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&v)[N])
    {
        float h = -INFINITY;
#pragma unroll
        for (int u = 0; u < N; ++u)
            h = fmaxf(fmaxf(h, fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y))),
                      fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
        return h;
    }
    static __device__ __forceinline__ uint4 pack(const float (&z)[PER])
    {
        return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
    }
};
struct LBF16 {
    using T = uint16_t;
    static constexpr int PER = 8;
    static constexpr uint32_t LOW = 0xff80ff80u;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(__ushort_as_bfloat16(v)); }
    static __device__ __forceinline__ T put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&z)[PER])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = __uint_as_float(w[i] << 16);
            z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&v)[N])
    {
        using P = __nv_bfloat162;
        const uint32_t low = LOW;
        P h = *reinterpret_cast<const P*>(&low);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) h = __hmax2(h, *reinterpret_cast<const P*>(&w[i]));
        }
        const float lo = __low2float(h), hi = __high2float(h);
        return fmaxf(lo, hi);
    }
    static __device__ __forceinline__ uint4 pack(const float (&z)[PER])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
struct LF16 {
    using T = uint16_t;
    static constexpr int PER = 8;
    static constexpr uint32_t LOW = 0xfc00fc00u;
    static __device__ __forceinline__ float get(T v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ T put(float v) { return __half_as_ushort(__float2half_rn(v)); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&z)[PER])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            z[2 * i] = f.x, z[2 * i + 1] = f.y;
        }
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&v)[N])
    {
        using P = __half2;
        const uint32_t low = LOW;
        P h = *reinterpret_cast<const P*>(&low);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) h = __hmax2(h, *reinterpret_cast<const P*>(&w[i]));
        }
        const float lo = __low2float(h), hi = __high2float(h);
        return fmaxf(lo, hi);
    }
    static __device__ __forceinline__ uint4 pack(const float (&z)[PER])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(z[2 * i], z[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Elements of a row before its first 16-byte boundary.
template <typename D>
__device__ __forceinline__ int head_of(const typename D::T* row, int V)
{
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(typename D::T);
    return min(V, off ? D::PER - off : 0);
}

// 1 / (T ln 2) as the exponents take it: t = (z h - reference(m, h)) c.
struct Scale {
    float h, c;
};
inline Scale scale_of(float temperature)
{
    const double c = 1.4426950408889634 / temperature;
    return c < 2. ? Scale{0.5f, (float)(2. * c)} : Scale{1.f, (float)c};
}

// m h of a largest logit; sums without a logit have the least finite one, from which -inf is -inf off.
__device__ __forceinline__ float reference(float m, float h) { return fmaxf(m, -FLT_MAX) * h; }

struct Sums {
    float m, s, q;  // largest logit, sum 2^t, sum 2^t t
};

// Everything relative to the larger m.  (s is one a logit at most: times 0 it is 0, or NaN where it was.)
template <bool ENT>
__device__ __forceinline__ Sums rescale(const Sums& a, float m, Scale by)
{
    if (a.m == m) return a;
    const float d = fmaxf((reference(a.m, by.h) - reference(m, by.h)) * by.c, FLOOR), f = ex2(d);
    return {m, a.s * f, ENT ? f * (a.q + d * a.s) : 0.f};
}
template <bool ENT>
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, Scale by)
{
    const float m = fmaxf(a.m, b.m);
    const Sums x = rescale<ENT>(a, m, by), y = rescale<ENT>(b, m, by);
    return {m, x.s + y.s, x.q + y.q};
}

__device__ __forceinline__ void st_cluster_u64(uint32_t at, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// A logit and its index as one number: larger ones first, equal ones by the lower index; 0: none.
// One key a lane, sorted over the warp, largest first (bitonic: every compare-exchange is of lanes
// 2^b apart).
__device__ __forceinline__ uint64_t exchange(uint64_t k, int d, bool larger)
{
    const uint64_t o = __shfl_xor_sync(0xffffffffu, k, d);
    return (k > o) == larger ? k : o;
}
__device__ __forceinline__ uint64_t sort_keys(uint64_t k)
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
        for (int d = n / 2; d > 0; d /= 2) k = exchange(k, d, ((lane & d) == 0) == ((lane & n) == 0 || n == 32));
    return k;
}
// The same with values alone (no NaN), and the 32 largest of two sorted warps of them, sorted.
__device__ __forceinline__ float exchange(float v, int d, bool larger)
{
    const float o = __shfl_xor_sync(0xffffffffu, v, d);
    return larger ? fmaxf(v, o) : fminf(v, o);
}
__device__ __forceinline__ float sort_values(float v)
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
        for (int d = n / 2; d > 0; d /= 2) v = exchange(v, d, ((lane & d) == 0) == ((lane & n) == 0 || n == 32));
    return v;
}
__device__ __forceinline__ float merge_values(float a, float b)
{
    const int lane = threadIdx.x % 32;
    float v = fmaxf(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v = exchange(v, d, (lane & d) == 0);
    return v;
}
// The 32 largest of two sorted warps of keys, sorted.
__device__ __forceinline__ uint64_t merge_best(uint64_t a, uint64_t b)
{
    const int lane = threadIdx.x % 32;
    const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
    uint64_t k = a > r ? a : r;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) k = exchange(k, d, (lane & d) == 0);
    return k;
}

struct LogprobsParams {
    const void* logits;
    int64_t ld;
    int V, top, cluster, threads;
    const int64_t* tokens;
    float inv_t;  // 1 / (T h)
    Scale by;
    float* logprobs;
    float* entropy;
    float* stats;
    float* top_logprobs;
    int64_t* top_tokens;
};

template <typename D, bool ENT, bool TOP>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(LogprobsParams p)
{
    constexpr int PER = D::PER;
    constexpr int LISTS = MAX_CLUSTER * WARPS;
    __shared__ float part_m[LISTS], part_s[LISTS], part_q[LISTS];
    __shared__ uint64_t lists_best[TOP ? LISTS : 1][TOP ? kMaxTop : 1];
    __shared__ uint64_t waiting[TOP ? WARPS : 1][TOP ? 64 : 1];
    __shared__ __align__(16) float high_of[TOP ? MAX_UNITS : 4];  // each unit's largest logit
    __shared__ uint16_t chosen[TOP ? MAX_UNITS : 1];              // units with the largest of them
    __shared__ int chosen_n;
    __shared__ float sorted_of[TOP ? WARPS : 1][TOP ? 32 : 1];  // each warp's units' largest
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = p.cluster, rank = blockIdx.x % C;
    const int64_t r = blockIdx.x / C;
    const int nthreads = blockDim.x, warps = nthreads / 32;
    if (TOP && threadIdx.x == 0) chosen_n = 0;
    if (C > 1) cluster_sync_all();  // (the first CTA's shared memory is written by the others)
    else if (TOP) __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();
    const typename D::T* row = static_cast<const typename D::T*>(p.logits) + r * p.ld;
    const Scale by = p.by;
    // the given token's logit, early
    float given = 0.f;
    bool have = false;
    if (rank == 0 && warp == 0) {
        const int64_t t = p.tokens[r];
        have = t >= 0 && t < p.V;
        if (have) given = D::get(row[t]);
    }
    const int head = head_of<D>(row, p.V);
    const int vecs = (p.V - head) / PER, tail0 = head + vecs * PER;
    const int v0 = (int)((int64_t)vecs * rank / C), v1 = (int)((int64_t)vecs * (rank + 1) / C);
    const uint4* body = reinterpret_cast<const uint4*>(row + head);

    Sums a = {-INFINITY, 0.f, 0.f};
    // a few elements outside the 16-byte vectors
    const auto edge = [&](int first, int n) {
        if ((int)threadIdx.x >= n) return;
        const float z = D::get(row[first + threadIdx.x]);
        if (z > a.m) a = rescale<ENT>(a, z, by);
        const float t = __fmaf_rn(z, by.h, -reference(a.m, by.h)) * by.c, e = ex2(t);
        a.s += e;
        if (ENT) a.q += e * fmaxf(t, FLOOR);
    };
    if (rank == 0 && head > 0) edge(0, head);

    // units: `in_row` next to each other in a row of vectors, the next ones `per_unit` batches on
    const int in_row = nthreads / 4, batch = FLY * nthreads;
    const int per_unit = TOP ? max(1, ((v1 - v0 + batch - 1) / batch + MAX_UNITS / in_row - 1) / (MAX_UNITS / in_row)) : 0;
    int units = 0, in_unit = 0;
    float unit_high = -INFINITY;
    const auto end_unit = [&] {
        unit_high = fmaxf(unit_high, __shfl_xor_sync(0xffffffffu, unit_high, 1));
        unit_high = fmaxf(unit_high, __shfl_xor_sync(0xffffffffu, unit_high, 2));
        if (lane % 4 == 0) high_of[units + threadIdx.x / 4] = unit_high;
        units += in_row, in_unit = 0, unit_high = -INFINITY;
    };

    uint4 next[FLY];
    const auto fetch = [&](int v) {
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            const int i = v + u * nthreads;
            next[u] = i < v1 ? __ldcs(body + i) : make_uint4(D::LOW, D::LOW, D::LOW, D::LOW);
        }
    };
    int v = v0 + (int)threadIdx.x;
    fetch(v);
    for (int b = v0; b < v1; b += batch, v += batch) {
        uint4 cur[FLY];
#pragma unroll
        for (int u = 0; u < FLY; ++u) cur[u] = next[u];
        if (b + batch < v1) fetch(v + batch);
        const float high = D::largest(cur);
        if constexpr (TOP) {
            unit_high = fmaxf(unit_high, high);
            if (++in_unit == per_unit) end_unit();
        }
        if (high > a.m) a = rescale<ENT>(a, high, by);
        const float ref = -reference(a.m, by.h);
        const float2 ref2 = make_float2(ref, ref), h2 = make_float2(by.h, by.h), c2 = make_float2(by.c, by.c);
        float2 s2 = make_float2(0.f, 0.f), q2 = s2;
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            float z[PER];
            D::unpack(cur[u], z);
#pragma unroll
            for (int j = 0; j < PER; j += 2) {
                float2 t = __fmul2_rn(__ffma2_rn(make_float2(z[j], z[j + 1]), h2, ref2), c2);
                const float2 e = make_float2(ex2(t.x), ex2(t.y));  // (NaN or inf where z is NaN or +inf)
                s2 = __fadd2_rn(s2, e);
                if (ENT) {
                    t.x = fmaxf(t.x, FLOOR), t.y = fmaxf(t.y, FLOOR);
                    q2 = __ffma2_rn(e, t, q2);
                }
            }
        }
        a.s += s2.x + s2.y;
        if (ENT) a.q += q2.x + q2.y;
    }
    if (rank == C - 1 && tail0 < p.V) edge(tail0, p.V - tail0);
    uint64_t best = 0;  // lane i: the warp's i-th best
    if constexpr (TOP) {
        // the units with the `top` largest maxima (more where they tie): all of the best in vectors are theirs
        if (in_unit > 0) end_unit();
        __syncthreads();
        float bound = -INFINITY;  // lane i: the i-th largest maximum, of the warp's units, then of all
        for (int u = threadIdx.x; u < units; u += nthreads) {  // (units are a multiple of 32)
            const float sorted = sort_values(high_of[u]);
            bound = u < nthreads ? sorted : merge_values(bound, sorted);
        }
        sorted_of[warp][lane] = bound;
        __syncthreads();
        bound = sorted_of[0][lane];
        for (int w = 1; w < min(warps, units / 32); ++w) bound = merge_values(bound, sorted_of[w][lane]);
        const float floor_v = __shfl_sync(0xffffffffu, bound, p.top - 1);  // `top` logits are no worse (-inf: read all)
        for (int u = threadIdx.x; u < units; u += nthreads) {
            const float high = high_of[u];
            const bool is = high >= floor_v && high > -INFINITY;
            const unsigned who = __ballot_sync(0xffffffffu, is);
            int first = 0;
            if (lane == 0 && who) first = atomicAdd(&chosen_n, __popc(who));
            first = __shfl_sync(0xffffffffu, first, 0);
            if (is) chosen[first + __popc(who & ((1u << lane) - 1))] = (uint16_t)u;
        }
        __syncthreads();
        const int n = chosen_n, each = per_unit * FLY;  // rows of four vectors of a unit
        uint64_t* const wait = waiting[warp];
        int pending = 0;
        float last = -INFINITY;  // the warp's top-th: its value and its index
        int last_i = -1;
        const auto flush = [&] {
            __syncwarp();
            const uint64_t sorted = sort_keys(lane < pending ? wait[lane] : 0ull);
            best = last_i == -1 ? sorted : merge_best(best, sorted);  // (-1: the first; all but a warp's last flush are of 32)
            __syncwarp();
            if (lane + 32 < pending) wait[lane] = wait[lane + 32];
            pending = max(pending - 32, 0);
            const uint64_t k = __shfl_sync(0xffffffffu, best, p.top - 1);
            last = key_value((uint32_t)(k >> 32));
            last_i = (int)~(uint32_t)k;
        };
        // a logit of each lane (-inf: none)
        const auto offer = [&](float v, int i) {
            const bool in = v >= floor_v && (v > last || (v == last && i < last_i));
            const unsigned w = __ballot_sync(0xffffffffu, in);
            if (w == 0) return;
            if (in) wait[pending + __popc(w & ((1u << lane) - 1))] = (uint64_t)order_key(v) << 32 | (uint32_t)~i;
            pending += __popc(w);
            if (pending >= 32) flush();
        };
        // their vectors once more, AHEAD vectors of a thread in flight
        constexpr int AHEAD = 4;
        const unsigned items = 4u * n * each;
        for (unsigned it0 = 0; it0 < items; it0 += AHEAD * nthreads) {
            uint4 w[AHEAD];
            int at[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const unsigned it = it0 + u * nthreads + threadIdx.x, j = it / 4, row = j / (unsigned)n;
                const int unit = it < items ? chosen[j - row * n] : 0;
                at[u] = it < items ? v0 + (unit / in_row * each + (int)row) * nthreads + (unit % in_row) * 4 + it % 4 : v1;
                w[u] = at[u] < v1 ? body[at[u]] : make_uint4(D::LOW, D::LOW, D::LOW, D::LOW);
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                float z[PER];
                D::unpack(w[u], z);
                unsigned mask = 0;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    mask |= z[j] >= floor_v && (z[j] > last || (z[j] == last && head + at[u] * PER + j < last_i)) ? 1u << j : 0u;
                // one of each lane's at a time
#pragma unroll 1
                while (__any_sync(0xffffffffu, mask != 0)) {
                    const int j = __ffs(mask) - 1;
                    float x = mask ? z[0] : -INFINITY;
#pragma unroll
                    for (int k = 1; k < PER; ++k) x = k == j ? z[k] : x;
                    offer(x, head + at[u] * PER + j);
                    mask &= mask - 1;
                }
            }
        }
        // and what lies outside the vectors
        if (warp == 0) {
            const int i = lane < 16 ? lane : tail0 + lane - 16;
            const bool in = lane < 16 ? rank == 0 && lane < head : rank == C - 1 && i < p.V;
            offer(in ? D::get(row[i]) : -INFINITY, i);
        }
        if (pending > 0) flush();
    }

    // the warps' sums and lists, at the first CTA
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        const Sums o = {__shfl_xor_sync(0xffffffffu, a.m, d), __shfl_xor_sync(0xffffffffu, a.s, d),
                          __shfl_xor_sync(0xffffffffu, a.q, d)};
        // (in the same order on both sides)
        a = (lane & d) ? join<ENT>(o, a, by) : join<ENT>(a, o, by);
    }
    const int list = rank * warps + warp;
    const auto at_first = [&](const void* q) { return C > 1 ? mapa_shared(smem_u32(q), 0) : smem_u32(q); };
    if (C > 1) {
        if (lane == 0) {
            st_shared_cluster_f32(at_first(&part_m[list]), a.m);
            st_shared_cluster_f32(at_first(&part_s[list]), a.s);
            if (ENT) st_shared_cluster_f32(at_first(&part_q[list]), a.q);
        }
        if (TOP && lane < p.top) st_cluster_u64(at_first(&lists_best[list][lane]), best);
        cluster_sync_all();
    } else {
        if (lane == 0) {
            part_m[list] = a.m, part_s[list] = a.s;
            if (ENT) part_q[list] = a.q;
        }
        if (TOP && lane < p.top) lists_best[list][lane] = best;
        __syncthreads();
    }
    if (rank != 0 || warp != 0) return;
    const int lists = C * warps;
    Sums t = {-INFINITY, 0.f, 0.f};
    for (int i = lane; i < lists; i += 32) {
        const Sums o = {part_m[i], part_s[i], ENT ? part_q[i] : 0.f};
        t = join<ENT>(t, o, by);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        const Sums o = {__shfl_xor_sync(0xffffffffu, t.m, d), __shfl_xor_sync(0xffffffffu, t.s, d),
                          __shfl_xor_sync(0xffffffffu, t.q, d)};
        t = (lane & d) ? join<ENT>(o, t, by) : join<ENT>(t, o, by);
    }
    float ln_s = t.m == INFINITY ? NAN : logf(t.s);
    const bool none = t.m == -INFINITY && t.s == 0.f;  // (a row of NaN has NaN sums)
    if (none) ln_s = 0.f;
    const auto logprob = [&](float z) { return __fmaf_rn(z, by.h, -t.m * by.h) * p.inv_t - ln_s; };
    if (lane == 0) {
        p.stats[2 * r] = t.m;
        p.stats[2 * r + 1] = ln_s;
        float lp = 0.f;
        if (have) lp = none ? -INFINITY : logprob(given);
        p.logprobs[r] = lp;
        if (ENT) p.entropy[r] = none ? 0.f : ln_s - LN2 * (t.q / t.s);
    }
    if constexpr (TOP) {
        // the best head of all lists, `top` times: a lane holds the heads of two lists
        const bool bad = ln_s != ln_s;
        int at0 = 0, at1 = 0;
        const auto head_key = [&](int l, int at) { return l < lists && at < p.top ? lists_best[l][at] : 0ull; };
        uint64_t key0 = head_key(lane, 0), key1 = head_key(lane + 32, 0), mine = 0;
        for (int j = 0; j < p.top && !bad; ++j) {
            const uint64_t k = key1 > key0 ? key1 : key0;
            const uint32_t m = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
            if (m == 0) break;
            const uint32_t i = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == m ? (uint32_t)k : 0u);
            const uint64_t w = (uint64_t)m << 32 | i;
            if (key0 == w) key0 = head_key(lane, ++at0);
            else if (key1 == w) key1 = head_key(lane + 32, ++at1);
            if (lane == j) mine = w;
        }
        const float val = key_value((uint32_t)(mine >> 32));
        const int64_t tok = mine ? (int64_t)(uint32_t)~(uint32_t)mine : -1;
        if (lane < p.top) {
            p.top_logprobs[r * p.top + lane] = bad ? ln_s : tok < 0 ? -INFINITY : logprob(val);
            p.top_tokens[r * p.top + lane] = tok;
        }
    }
}

// ------------------------------------------------------------------ gradient

struct LogprobsGradParams {
    const void* logits;
    int64_t ld;
    int V, blocks;  // blocks of a row
    const int64_t* tokens;
    float inv_t;
    Scale by;
    const float* stats;
    const float* entropy;
    const float* dlogprobs;
    const float* dentropy;
    void* dlogits;
    int64_t ldd;
};

constexpr int GRAD_FLY = 4;

// dz_j = (g (delta_jt - p_j) - h p_j (ln p_j + H)) / T = p_j (A + B log2 p_j) + delta_jt g / T,
// log2 p_j = t_j - ln S / ln 2
template <typename D, bool ENT>
__global__ void __launch_bounds__(THREADS) logprobs_grad_kernel(LogprobsGradParams p)
{
    constexpr int PER = D::PER;
    using T = typename D::T;
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t r = blockIdx.x / p.blocks;
    const int part = blockIdx.x % p.blocks;
    const T* row = static_cast<const T*>(p.logits) + r * p.ld;
    T* out = static_cast<T*>(p.dlogits) + r * p.ldd;
    const int64_t tok = p.tokens[r];
    const float m = p.stats[2 * r], ln_s = p.stats[2 * r + 1];
    const Scale by = p.by;
    const bool have = tok >= 0 && tok < p.V;
    const float g = have && p.dlogprobs ? p.dlogprobs[r] : 0.f, h = ENT ? p.dentropy[r] : 0.f;
    const bool zero = (g == 0.f && h == 0.f) || (m == -INFINITY && ln_s == ln_s);
    const float B = -h * p.inv_t * LN2, A = ENT ? -(g + h * p.entropy[r]) * p.inv_t : -g * p.inv_t;
    const float gt = g * p.inv_t;
    // g / T or h / T about as large as fp32's values go (B times an exponent no less): 1 / T comes last then, as p may
    // bring the product back, to 0 above all
    const bool large = !(fabsf(A) < 1e33f && fabsf(B) < 1e33f && fabsf(gt) < 1e33f);
    const int t = have ? (int)tok : -1;
    const float ref = reference(m, by.h), log_s = ln_s * LOG2E;
    const auto grad = [&](float z, int j) {
        if (zero) return 0.f;
        if (ln_s != ln_s) return ln_s;  // a row with NaN
        const float l = __fmaf_rn(__fmaf_rn(z, by.h, -ref), by.c, -log_s);
        const float e = ex2(l);
        if (large) {
            const float v = -e * g - (ENT ? e * h * (p.entropy[r] + LN2 * fmaxf(l, FLOOR)) : 0.f);
            return (j == t ? v + g : v) * p.inv_t;
        }
        const float v = ENT ? e * (A + B * fmaxf(l, FLOOR)) : e * A;
        return j == t ? v + gt : v;
    };
    const int head = head_of<D>(row, p.V), vecs = (p.V - head) / PER;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out + head)) & 15) == 0;
    if (!aligned || large || ln_s != ln_s) {
        const int n = (p.V + p.blocks - 1) / p.blocks, j1 = min(p.V, (part + 1) * n);
        for (int j = part * n + (int)threadIdx.x; j < j1; j += THREADS)
            out[j] = D::put(grad(zero ? 0.f : D::get(row[j]), j));
        return;
    }
    const int v0 = (int)((int64_t)vecs * part / p.blocks), v1 = (int)((int64_t)vecs * (part + 1) / p.blocks);
    const uint4* src = reinterpret_cast<const uint4*>(row + head);
    uint4* dst = reinterpret_cast<uint4*>(out + head);
    if (zero) {
        for (int v = v0 + (int)threadIdx.x; v < v1; v += THREADS) __stcs(dst + v, make_uint4(0, 0, 0, 0));
    } else {
        const float2 h2 = make_float2(by.h, by.h), c2 = make_float2(by.c, by.c);
        const float2 ref2 = make_float2(-ref, -ref), log2 = make_float2(-log_s, -log_s);
        const float2 A2 = make_float2(A, A), B2 = make_float2(B, B);
        for (int v = v0 + (int)threadIdx.x; v < v1; v += GRAD_FLY * THREADS) {
            uint4 in[GRAD_FLY];
#pragma unroll
            for (int u = 0; u < GRAD_FLY; ++u)
                if (v + u * THREADS < v1) in[u] = __ldcs(src + v + u * THREADS);
#pragma unroll
            for (int u = 0; u < GRAD_FLY; ++u) {
                if (v + u * THREADS >= v1) break;
                float z[PER];
                D::unpack(in[u], z);
#pragma unroll
                for (int j = 0; j < PER; j += 2) {
                    float2 l = __ffma2_rn(__ffma2_rn(make_float2(z[j], z[j + 1]), h2, ref2), c2, log2);
                    const float2 e = make_float2(ex2(l.x), ex2(l.y));
                    float2 w = A2;
                    if (ENT) {
                        l.x = fmaxf(l.x, FLOOR), l.y = fmaxf(l.y, FLOOR);
                        w = __ffma2_rn(B2, l, A2);
                    }
                    const float2 d = __fmul2_rn(e, w);
                    z[j] = d.x, z[j + 1] = d.y;
                }
                const unsigned at = (unsigned)(t - (head + (v + u * THREADS) * PER));
                if (at < (unsigned)PER)
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (j == (int)at) z[j] += gt;
                __stcs(dst + v + u * THREADS, D::pack(z));
            }
        }
    }
    if (part == 0 && (int)threadIdx.x < head)
        out[threadIdx.x] = D::put(grad(zero ? 0.f : D::get(row[threadIdx.x]), threadIdx.x));
    const int tail = head + vecs * PER + (int)threadIdx.x;
    if (part == p.blocks - 1 && tail < p.V) out[tail] = D::put(grad(zero ? 0.f : D::get(row[tail]), tail));
}

template <typename D, bool ENT, bool TOP>
cudaError_t launch_rows(const LogprobsParams& p, int64_t rows, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cluster), 1, 1);
    cfg.blockDim = dim3(p.threads, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<D, ENT, TOP>, p);
}

template <typename D>
cudaError_t launch_typed(const LogprobsParams& p, int64_t rows, cudaStream_t s)
{
    if (p.entropy) return p.top > 0 ? launch_rows<D, true, true>(p, rows, s) : launch_rows<D, true, false>(p, rows, s);
    return p.top > 0 ? launch_rows<D, false, true>(p, rows, s) : launch_rows<D, false, false>(p, rows, s);
}

template <typename D>
cudaError_t launch_grad_typed(const LogprobsGradParams& p, int64_t rows, cudaStream_t s)
{
    const dim3 grid((unsigned)(rows * p.blocks)), block(THREADS);
    return p.dentropy ? launch_dependent(logprobs_grad_kernel<D, true>, grid, block, 0, s, p)
                      : launch_dependent(logprobs_grad_kernel<D, false>, grid, block, 0, s, p);
}

}  // namespace

int launch_logprobs(const LogprobsArgs& a, int num_sms, cudaStream_t s, int* launches)
{
    LogprobsParams p = {};
    p.logits = a.logits, p.ld = a.ld;
    p.V = a.V, p.top = a.top;
    p.tokens = a.tokens;
    p.by = scale_of(a.temperature);
    p.inv_t = (float)(1. / p.by.h / a.temperature);
    p.logprobs = a.logprobs, p.entropy = a.entropy, p.stats = a.stats;
    p.top_logprobs = a.top_logprobs, p.top_tokens = a.top_tokens;
    const int batch = FLY * THREADS / 2 * 16 / (a.dtype == GEMM_F32 ? 4 : 2);
    // CTAs a row: as many as are resident at once (nine an SM, by their registers) and have two batches
    // to read
    p.cluster = 1;
    while (p.cluster < MAX_CLUSTER && a.rows * 2 * p.cluster <= 9 * (int64_t)num_sms && a.V > p.cluster * batch)
        p.cluster *= 2;
    // Four warps a CTA: more of them are resident and less of the last wave is idle.  Eight where long rows
    // do not fill the SMs and the loads in flight count.  us with four and eight warps (bf16, entropy):
    //   4000 x 12000 28 45, 2000 x 50257 43 53, 4096 x 131072 162 168; 1000 x 131072 52 49
    const int few = THREADS / 2;
    p.threads = a.rows * p.cluster < 8 * (int64_t)num_sms && a.V / p.cluster > 1 << 16 ? THREADS : few;
    const cudaError_t e = a.dtype == GEMM_F32    ? launch_typed<LF32>(p, a.rows, s)
                          : a.dtype == GEMM_BF16 ? launch_typed<LBF16>(p, a.rows, s)
                                                 : launch_typed<LF16>(p, a.rows, s);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

int launch_logprobs_grad(const LogprobsGradArgs& a, cudaStream_t s, int* launches)
{
    LogprobsGradParams p = {};
    p.logits = a.logits, p.ld = a.ld;
    p.V = a.V;
    // a batch of loads a block
    const int batch = GRAD_FLY * THREADS * 16 / (a.dtype == GEMM_F32 ? 4 : 2);
    p.blocks = (a.V + batch - 1) / batch;
    p.tokens = a.tokens;
    p.inv_t = 1.f / a.temperature;
    p.by = scale_of(a.temperature);
    p.stats = a.stats, p.entropy = a.entropy;
    p.dlogprobs = a.dlogprobs, p.dentropy = a.dentropy;
    p.dlogits = a.dlogits, p.ldd = a.ldd;
    if (a.rows * p.blocks > 0x7fffffffLL) return GEMM_ERR_UNSUPPORTED;
    const cudaError_t e = a.dtype == GEMM_F32    ? launch_grad_typed<LF32>(p, a.rows, s)
                          : a.dtype == GEMM_BF16 ? launch_grad_typed<LBF16>(p, a.rows, s)
                                                 : launch_grad_typed<LF16>(p, a.rows, s);
    if (e != cudaSuccess) return GEMM_ERR_CUDA;
    *launches += 1;
    return GEMM_OK;
}

}  // namespace gemm_gb300
