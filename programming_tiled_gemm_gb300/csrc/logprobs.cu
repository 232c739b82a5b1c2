// Log probabilities of given tokens, the entropy and the best alternatives of rows of logits,
// and the logits' gradient.
//
// With u_j = (z_j - m) / T, m the row's largest logit: S = sum exp(u_j), ln p_j = u_j - ln S,
// H = ln S - sum exp(u_j) u_j / S.  One pass: every thread keeps its own m, S and Q = sum
// exp(u) u (in units of ln 2, for ex2) and rescales them when m grows,
//     S' = f S,  Q' = f (Q + d S),  d = (m - m') / T,  f = exp(d),
// and the threads' triples are joined the same way.  u is taken as (z - m) times 1 / T, never as
// z / T - m / T: that loses what the two share and overflows at the type's lowest value.  As a
// factor of exp(u), u is clamped at -1e4, far below where exp is 0: 0 * -inf is 0 there.
//
// Alternatives: a warp keeps the `top` best it has seen, one a lane, in order.  A logit is looked
// at only if it beats the warp's last one and is no worse than a bound that all warps of the CTA
// raise; a first bound is the top-th largest of the lanes' maxima of the first batch (at least
// `top` logits are no worse), so some `top` insertions a warp remain.  A warp meets its logits in
// the order of their index, so equal ones keep that order.
//
// A cluster of up to 8 CTAs shares a row where there are few (their sums and lists go to the
// first CTA's shared memory); rows are read with 16-byte loads from the first 16-byte boundary
// on, wherever they start.  One launch each, no workspace, sums in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "logprobs.h"
#include "ptx.h"

namespace gemm_gb300 {

namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int MAX_CLUSTER = 8;
constexpr int FLY = 4;  // 16-byte loads of a thread in a batch
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

struct Triple {
    float m, s, q;  // largest logit, sum exp(u), sum exp(u) u / ln 2, with u = (z - m) / T
};

// Everything relative to the larger m.
template <bool ENT>
__device__ __forceinline__ Triple rescale(const Triple& a, float m, float c)
{
    if (a.m == m || a.m == -INFINITY) return {m, a.s, a.q};  // (without logits there is nothing to scale)
    const float d = fmaxf((a.m - m) * c, FLOOR), f = ex2(d);
    return {m, a.s * f, ENT ? f * (a.q + d * a.s) : 0.f};
}
template <bool ENT>
__device__ __forceinline__ Triple join(const Triple& a, const Triple& b, float c)
{
    const float m = fmaxf(a.m, b.m);
    const Triple x = rescale<ENT>(a, m, c), y = rescale<ENT>(b, m, c);
    return {m, x.s + y.s, x.q + y.q};
}

__device__ __forceinline__ void st_cluster_f32(uint32_t at, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t at, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

struct LogprobsParams {
    const void* logits;
    int64_t ld;
    int V, top, cluster;
    const int64_t* tokens;
    float inv_t, c;  // 1 / T and 1 / (T ln 2)
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
    __shared__ float list_v[TOP ? LISTS : 1][TOP ? kMaxTop : 1];
    __shared__ uint32_t list_i[TOP ? LISTS : 1][TOP ? kMaxTop : 1];
    __shared__ uint32_t bound;  // a key: `top` logits of the row are no worse
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = p.cluster, rank = blockIdx.x % C;
    const int64_t r = blockIdx.x / C;
    if (TOP && threadIdx.x == 0) bound = 0;
    if (C > 1) cluster_sync_all();  // (the first CTA's shared memory is written by the others)
    else if (TOP) __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();
    const typename D::T* row = static_cast<const typename D::T*>(p.logits) + r * p.ld;
    const float c = p.c;
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

    Triple a = {-INFINITY, 0.f, 0.f};
    // the warp's best: lane i the i-th
    float best = -INFINITY;
    int best_i = -1;
    float last = -INFINITY;  // the top-th, in every lane
    float floor_v = -INFINITY;
    const auto insert = [&](float v, int i) {
        const int at = __popc(__ballot_sync(0xffffffffu, best >= v));  // (equal ones came earlier: lower indices)
        const float up = __shfl_up_sync(0xffffffffu, best, 1);
        const int up_i = __shfl_up_sync(0xffffffffu, best_i, 1);
        if (lane > at) best = up, best_i = up_i;
        if (lane == at) best = v, best_i = i;
        last = __shfl_sync(0xffffffffu, best, p.top - 1);
    };
    // N logits of each lane, in the order of the lanes
    const auto offer = [&](const auto& z, int first, int n) {
        constexpr int N = sizeof(z) / sizeof(float);
        for (;;) {
            unsigned mask = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) mask |= (j < n && z[j] > last && z[j] >= floor_v) ? 1u << j : 0u;
            const unsigned who = __ballot_sync(0xffffffffu, mask != 0);
            if (who == 0) break;
            const int src = __ffs(who) - 1;
            // that lane's candidates in order; each is taken off before the next look
            unsigned left = __shfl_sync(0xffffffffu, mask, src);
            while (left) {
                const int j = __ffs(left) - 1;
                left &= left - 1;
                float v = z[0];
#pragma unroll
                for (int k = 1; k < N; ++k)
                    if (k == j) v = z[k];
                v = __shfl_sync(0xffffffffu, v, src);
                if (v > last) insert(v, __shfl_sync(0xffffffffu, first, src) + j);
            }
            if (lane <= src) n = 0;  // those before it had none
        }
    };
    const auto add = [&](float z, float m) {
        const float t = (z - m) * c, e = ex2(t);  // (NaN where z is NaN or +inf)
        a.s += e;
        if (ENT) a.q += e * fmaxf(t, FLOOR);
    };
    // a few elements outside the 16-byte vectors
    const auto edge = [&](int first, int n) {
        float z[1] = {(int)threadIdx.x < n ? D::get(row[first + threadIdx.x]) : -INFINITY};
        if ((int)threadIdx.x < n) {
            if (z[0] > a.m) a = rescale<ENT>(a, z[0], c);
            add(z[0], a.m == -INFINITY ? 0.f : a.m);
        }
        if (TOP && warp == 0) offer(z, first + (int)threadIdx.x, (int)threadIdx.x < n);
    };
    if (rank == 0 && head > 0) edge(0, head);

    uint4 next[FLY];
    const auto fetch = [&](int v) {
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            const int i = v + u * THREADS;
            next[u] = i < v1 ? __ldcs(body + i) : make_uint4(D::LOW, D::LOW, D::LOW, D::LOW);
        }
    };
    bool begun = false;
    int v = v0 + (int)threadIdx.x;
    fetch(v);
    for (int b = v0; b < v1; b += FLY * THREADS, v += FLY * THREADS) {
        uint4 cur[FLY];
#pragma unroll
        for (int u = 0; u < FLY; ++u) cur[u] = next[u];
        if (b + FLY * THREADS < v1) fetch(v + FLY * THREADS);
        float high = -INFINITY;
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            float z[PER];
            D::unpack(cur[u], z);
#pragma unroll
            for (int j = 0; j < PER; ++j) high = fmaxf(high, z[j]);
        }
        if (high > a.m) a = rescale<ENT>(a, high, c);
        const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            float z[PER];
            D::unpack(cur[u], z);
#pragma unroll
            for (int j = 0; j < PER; ++j) add(z[j], m);
        }
        if (TOP) {
            if (!begun) {
                // the top-th largest of the lanes' maxima
                begun = true;
                int better = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float o = __shfl_sync(0xffffffffu, high, i);
                    better += o > high || (o == high && i < lane);
                }
                const float kth = __shfl_sync(0xffffffffu, high,
                                              __ffs(__ballot_sync(0xffffffffu, better == p.top - 1)) - 1);
                if (lane == 0) atomicMax(&bound, order_key(kth));
                floor_v = kth;
            }
            floor_v = fmaxf(floor_v, key_value(*(volatile uint32_t*)&bound));
            if (__any_sync(0xffffffffu, high > last && high >= floor_v)) {
#pragma unroll
                for (int u = 0; u < FLY; ++u) {
                    float z[PER];
                    D::unpack(cur[u], z);
                    offer(z, head + (v + u * THREADS) * PER, v + u * THREADS < v1 ? PER : 0);
                }
                if (lane == 0 && last > -INFINITY) atomicMax(&bound, order_key(last));
            }
        }
    }
    if (rank == C - 1 && tail0 < p.V) edge(tail0, p.V - tail0);

    // the warps' sums and lists, at the first CTA
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        const Triple o = {__shfl_xor_sync(0xffffffffu, a.m, d), __shfl_xor_sync(0xffffffffu, a.s, d),
                          __shfl_xor_sync(0xffffffffu, a.q, d)};
        // (in the same order on both sides)
        a = (lane & d) ? join<ENT>(o, a, c) : join<ENT>(a, o, c);
    }
    const int list = rank * WARPS + warp;
    const auto at0 = [&](const void* q) { return C > 1 ? mapa_shared(smem_u32(q), 0) : smem_u32(q); };
    if (C > 1) {
        if (lane == 0) {
            st_cluster_f32(at0(&part_m[list]), a.m);
            st_cluster_f32(at0(&part_s[list]), a.s);
            if (ENT) st_cluster_f32(at0(&part_q[list]), a.q);
        }
        if (TOP && lane < p.top) {
            st_cluster_f32(at0(&list_v[list][lane]), best);
            st_cluster_u32(at0(&list_i[list][lane]), (uint32_t)best_i);
        }
        cluster_sync_all();
    } else {
        if (lane == 0) {
            part_m[list] = a.m, part_s[list] = a.s;
            if (ENT) part_q[list] = a.q;
        }
        if (TOP && lane < p.top) list_v[list][lane] = best, list_i[list][lane] = (uint32_t)best_i;
        __syncthreads();
    }
    if (rank != 0 || warp != 0) return;
    const int lists = C * WARPS;
    Triple t = {-INFINITY, 0.f, 0.f};
    for (int i = lane; i < lists; i += 32) {
        const Triple o = {part_m[i], part_s[i], ENT ? part_q[i] : 0.f};
        t = join<ENT>(t, o, c);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        const Triple o = {__shfl_xor_sync(0xffffffffu, t.m, d), __shfl_xor_sync(0xffffffffu, t.s, d),
                          __shfl_xor_sync(0xffffffffu, t.q, d)};
        t = (lane & d) ? join<ENT>(o, t, c) : join<ENT>(t, o, c);
    }
    const bool none = t.m == -INFINITY && t.s == 0.f;  // (a row of NaN has NaN sums)
    const float ln_s = none ? 0.f : logf(t.s);
    if (lane == 0) {
        p.stats[2 * r] = t.m;
        p.stats[2 * r + 1] = ln_s;
        float lp = 0.f;
        if (have) lp = none ? -INFINITY : (given - t.m) * p.inv_t - ln_s;
        p.logprobs[r] = lp;
        if (ENT) p.entropy[r] = none ? 0.f : ln_s - LN2 * (t.q / t.s);
    }
    if constexpr (TOP) {
        // the best head of all lists, `top` times: a lane holds the heads of two lists
        const bool bad = ln_s != ln_s;
        uint32_t key[2], idx[2];
        int at[2] = {0, 0};
        const auto head_key = [&](int h) {
            const int l = lane + 32 * h;
            const bool in = l < lists && at[h] < p.top;
            key[h] = in ? order_key(list_v[l][at[h]]) : 0u;
            idx[h] = in ? list_i[l][at[h]] : 0xffffffffu;
        };
        head_key(0);
        head_key(1);
        float val = -INFINITY;
        int64_t tok = -1;
        for (int j = 0; j < p.top && !bad; ++j) {
            const int h = key[1] > key[0] || (key[1] == key[0] && idx[1] < idx[0]);
            const uint32_t k = h ? key[1] : key[0], i = h ? idx[1] : idx[0];
            const uint32_t m = __reduce_max_sync(0xffffffffu, k);
            if (m == 0) break;
            const uint32_t w = __reduce_min_sync(0xffffffffu, k == m ? i : 0xffffffffu);
            if (k == m && i == w) {
                ++at[h];
                head_key(h);
            }
            if (lane == j) val = key_value(m), tok = (int64_t)w;
        }
        if (lane < p.top) {
            p.top_logprobs[r * p.top + lane] = bad ? ln_s : tok < 0 ? -INFINITY : (val - t.m) * p.inv_t - ln_s;
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
    const float* stats;
    const float* entropy;
    const float* dlogprobs;
    const float* dentropy;
    void* dlogits;
    int64_t ldd;
};

constexpr int GRAD_FLY = 4;

// dz_j = (g (delta_jt - p_j) - h p_j (ln p_j + H)) / T = p_j (A + B ln p_j) + delta_jt g / T
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
    const bool have = tok >= 0 && tok < p.V;
    const float g = have && p.dlogprobs ? p.dlogprobs[r] : 0.f, h = ENT ? p.dentropy[r] : 0.f;
    const bool zero = (g == 0.f && h == 0.f) || (m == -INFINITY && ln_s == ln_s);
    const float B = -h * p.inv_t, A = ENT ? -(g + h * p.entropy[r]) * p.inv_t : -g * p.inv_t;
    const float gt = g * p.inv_t;
    const int t = have ? (int)tok : -1;
    const auto grad = [&](float z, int j) {
        if (zero) return 0.f;
        const float l = fmaxf((z - m) * p.inv_t - ln_s, FLOOR);
        // (16-bit results: l * log2 e rounds by 2^-24 |l|, far below theirs)
        const float e = PER == 4 ? expf(l) : ex2(l * LOG2E);
        const float v = ENT ? e * (A + B * l) : e * A;
        return j == t ? v + gt : v;
    };
    const int head = head_of<D>(row, p.V), vecs = (p.V - head) / PER;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out + head)) & 15) == 0;
    const int n = (p.V + p.blocks - 1) / p.blocks;  // (unaligned: elements of this block)
    const bool bad = ln_s != ln_s;                   // a row with NaN: all of it
    if (!aligned || bad) {
        const int j1 = min(p.V, (part + 1) * n);
        for (int j = part * n + (int)threadIdx.x; j < j1; j += THREADS)
            out[j] = D::put(bad && !zero ? ln_s : grad(zero ? 0.f : D::get(row[j]), j));
        return;
    }
    const int v0 = (int)((int64_t)vecs * part / p.blocks), v1 = (int)((int64_t)vecs * (part + 1) / p.blocks);
    const uint4* src = reinterpret_cast<const uint4*>(row + head);
    uint4* dst = reinterpret_cast<uint4*>(out + head);
    for (int v = v0 + (int)threadIdx.x; v < v1; v += GRAD_FLY * THREADS) {
        uint4 in[GRAD_FLY];
        if (!zero) {
#pragma unroll
            for (int u = 0; u < GRAD_FLY; ++u)
                if (v + u * THREADS < v1) in[u] = __ldcs(src + v + u * THREADS);
        }
#pragma unroll
        for (int u = 0; u < GRAD_FLY; ++u) {
            if (v + u * THREADS >= v1) break;
            float z[PER];
            if (zero) in[u] = make_uint4(0, 0, 0, 0);
            D::unpack(in[u], z);
            const int j0 = head + (v + u * THREADS) * PER;
#pragma unroll
            for (int j = 0; j < PER; ++j) z[j] = grad(z[j], j0 + j);
            __stcs(dst + v + u * THREADS, D::pack(z));
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
    cfg.blockDim = dim3(THREADS, 1, 1);
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
    p.inv_t = 1.f / a.temperature;
    p.c = (float)(1.4426950408889634 / a.temperature);
    p.logprobs = a.logprobs, p.entropy = a.entropy, p.stats = a.stats;
    p.top_logprobs = a.top_logprobs, p.top_tokens = a.top_tokens;
    // CTAs a row: as many as are resident at once (six an SM) and have a batch to read
    const int batch = FLY * THREADS * 16 / (a.dtype == GEMM_F32 ? 4 : 2);
    p.cluster = 1;
    while (p.cluster < MAX_CLUSTER && a.rows * 2 * p.cluster <= 6 * (int64_t)num_sms && a.V > p.cluster * batch / 2)
        p.cluster *= 2;
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
