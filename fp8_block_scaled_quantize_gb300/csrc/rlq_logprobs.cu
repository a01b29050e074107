// Token log probabilities with entropy and the most likely alternatives, and the gradient of any
// loss of log probabilities and entropy with respect to the logits (sm_103a).
//
// Per row of logits x [V] with target t, z = x / temperature, m its maximum:
//   S = sum_v exp(z_v - m),  lse = m + log S,  lp = z_t - lse
//   H = -sum_v p_v log p_v = log S - sum_v exp(z_v - m) (z_v - m) / S
//   the k largest logits, among equal ones the lowest token, and their log probabilities
//   dx_v = ([v = t] dlp - p_v (dlp + dH (log p_v + H))) / temperature,  p_v = exp(z_v - lse)
// Both terms of H are >= 0, so nothing cancels; a logit of -inf adds nothing to either sum.
//
// Forward, bound by memory (the logits are read once): a CTA (few rows: a cluster, a part each)
// streams its row with running maximum, sum and weighted sum a thread.  The alternatives cost
// the loop nothing: it keeps each thread's maximum anyway.  The k-th largest of those T is a
// lower bound of the row's k-th logit, so every wanted logit is in one of the few threads whose
// maximum reaches T, as a rule in the batch of loads that the maximum is in; those batches are
// read again, and what reaches T goes on a list, whose ranks are counted.  A list that
// overflows (thousands of equal logits) is replaced by a search for the k-th logit over the
// whole row, some 35 passes over it.  Masks of -inf never come to that; masks that are numbers
// (-10^9, the type's lowest value) do in rows that leave fewer tokens than alternatives: 600 x 32001
// fp32, 20 alternatives, one to ten tokens left: 20 us under -inf, 650-690 under such masks.
//
// Measured: 2048 x 128256 bf16 with 20 alternatives 102 us (0.76 of HBM; without them 88, a row's
// end and the batches read again, some of which L2 no longer has, are the rest), 1000 x
// 128256 fp32 88 (0.86), 64 x 151936 bf16 12.8, 1 x 128256 7.6 (3.4 without alternatives: a
// chain of barriers and loads).  Reading all units of a chosen thread again took 133 and 125 us
// for the first two.  512 threads a CTA: 113 us; a bound on the maxima of 2 k + 8 threads: 104.
//
// Backward, bound by memory (read once, written once): lse and H come from the forward pass, so a
// unit's gradient needs nothing but the unit and the row's factors.  4096 x 128256 bf16, 15% of
// the rows empty and not read: 283 us (1.01 of the copy rate); 600 x 32001 fp32 25 (0.90).  Rows whose
// |lse| is above 256 are formed by one CTA in three passes: 64 x 128256 bf16 102 us, 8.7 otherwise.
#include <cuda_runtime.h>

#include "rlq_internal.h"
#include "rlq_rows.cuh"

namespace rlq {
namespace {

constexpr float LN2 = 0.6931471805599453f;
constexpr float LOWEST = -16384.0f;  // 2^LOWEST is 0, and 0 x LOWEST too

constexpr int THREADS = 256, CTAS_SM = 4, WARPS = THREADS / 32, MAX_CLUSTER = 8;
static_assert((THREADS & (THREADS - 1)) == 0, "a batch's number and a thread's share a word");
constexpr int BATCH = 8;     // 16-byte loads in flight a thread
constexpr int MAX_TOP = MAX_TOKEN_TOP;
constexpr int LIST = 1024;   // candidates
constexpr int CHOSEN = 1024; // batches read again

struct Sums {
    float m, s, w;  // maximum, sum of 2^t and of t 2^t, t = (x - m) c
};

// The lanes' sums, joined in every lane.  Sums of -inf only are 0; one that met a NaN is NaN.
__device__ __forceinline__ Sums join(Sums v, float c)
{
    float m = v.m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float s = 0.0f, w = 0.0f;
    if (v.s != 0.0f) {
        const float d = (v.m - m) * c, k = ex2(d);
        s = v.s * k;
        w = k == 0.0f ? 0.0f : fmaf(d, v.s, v.w) * k;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
    }
    return {m, s, w};
}

// m / temperature + ls, rounded once but for ls's last place: the reciprocal is the sum of two floats
// (rounded to one, it takes up to 2^-24 of m / temperature more, and every probability that the
// gradient forms of the lse with it: 1.4e-5 next to 256).
__device__ __forceinline__ float lse_of(float m, float ls, float inv_hi, float inv_lo)
{
    const float z = m * inv_hi;
    // (where that overflows, the low part's product would be an infinity of its own sign)
    return fabsf(z) < INFINITY ? fmaf(m, inv_hi, fmaf(m, inv_lo, ls)) : z + ls;
}

// Unsigned integers in the order of the floats, and back (what lies below -inf is -inf).
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k)
{
    return k <= 0x007FFFFFu ? -INFINITY : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Whether logit a at token i comes before b at token j.
__device__ __forceinline__ bool before(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

// What a CTA has of its row, and the row's units.
template <typename T>
struct Part {
    const T *x;
    int V, off, u0, u1, whole0, whole1;  // as in the loss's kernel: unit u is elements u N - off ..
    __device__ __forceinline__ uint4 load(int u) const
    {
        constexpr uint32_t NINF = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
        if (u >= u1)
            return make_uint4(NINF, NINF, NINF, NINF);
        return u >= whole0 && u < whole1 ? ld_row(x + ((int64_t)u * Elem<T>::N - off)) : load_cut(x, u * Elem<T>::N - off, V);
    }
    // f(value, token) for each of a unit's elements that exists
    template <typename F>
    __device__ __forceinline__ void each(int u, F f) const
    {
        if (u < u1)
            each_of(load(u), u, f);
    }
    template <typename F>
    __device__ __forceinline__ void each_of(const uint4 &v, int u, F f) const
    {
        if (u >= u1)
            return;
        const int e0 = u * Elem<T>::N - off;
#pragma unroll
        for (int j = 0; j < Elem<T>::N; j += 2) {
            const float2 e = Elem<T>::get2(v, j / 2);
            if (e0 + j >= 0 && e0 + j < V)
                f(e.x, e0 + j);
            if (e0 + j + 1 >= 0 && e0 + j + 1 < V)
                f(e.y, e0 + j + 1);
        }
    }
};

struct Candidates {
    float x[LIST];
    int at[LIST];
    int n;          // candidates, also those past the list's end
    int n_chosen;
    int chosen[CHOSEN];  // batch x THREADS + thread
    int scratch[WARPS + 1];
    float thread_max[THREADS];
};

__device__ __forceinline__ void put(Candidates &c, float x, int at)
{
    const int i = atomicAdd(&c.n, 1);
    if (i < LIST) {
        c.x[i] = x;
        c.at[i] = at;
    }
}

// Sum over the CTA, in every thread.
__device__ __forceinline__ int cta_sum(Candidates &c, int v)
{
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        c.scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i)
        s += c.scratch[i];
    return s;
}

// The first `want` tokens, in order, whose logit equals `value`.
template <typename T>
__device__ __noinline__ void put_first_equal(const Part<T> &p, Candidates &c, float value, int want)
{
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x / 32;
    int have = 0;
    for (int base = p.u0; base < p.u1 && have < want; base += blockDim.x) {
        int mine = 0;
        p.each(base + t, [&](float x, int) { mine += x == value; });
        int before_me = mine;  // inclusive scan over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, before_me, o);
            before_me += lane >= o ? y : 0;
        }
        __syncthreads();
        if (lane == 31)
            c.scratch[warp] = before_me;
        __syncthreads();
        int at = have + before_me - mine;
        for (int i = 0; i < nw; ++i) {
            at += i < warp ? c.scratch[i] : 0;
            have += c.scratch[i];
        }
        p.each(base + t, [&](float x, int token) {
            if (x == value && at++ < want)
                put(c, x, token);
        });
    }
}

// The list overflowed: the k-th largest logit by bisection between `low`, which k logits
// reach, and `high`, which none exceeds; then the logits above it and the first equal ones.
template <typename T>
__device__ __noinline__ void search(const Part<T> &p, Candidates &c, float low, float high, int k)
{
    uint32_t lo = key_of(low), hi = key_of(high);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const float v = of_key(mid);
        int mine = 0;
        for (int u = p.u0 + threadIdx.x; u < p.u1; u += blockDim.x)
            p.each(u, [&](float x, int) { mine += x >= v; });
        if (cta_sum(c, mine) >= k)
            lo = mid;
        else
            hi = mid - 1;
    }
    const float v = of_key(lo);
    __syncthreads();
    if (threadIdx.x == 0)
        c.n = 0;
    __syncthreads();
    for (int u = p.u0 + threadIdx.x; u < p.u1; u += blockDim.x)
        p.each(u, [&](float x, int token) {
            if (x > v)
                put(c, x, token);
        });
    __syncthreads();
    const int above = c.n;
    __syncthreads();
    put_first_equal(p, c, v, k - above);
}

// T, a value that at least k of the threads' maxima reach and, unless equal ones stand in the
// way, at most 5/4 k + 2 (by one warp): bisection of the keys between the smallest and the largest.
__device__ __forceinline__ float threshold(const float *thread_max, int lane, int k)
{
    uint32_t key[WARPS], lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const bool in = 32 * i + lane < (int)blockDim.x;
        key[i] = in ? key_of(thread_max[32 * i + lane]) : 0u;
        lo = min(lo, in ? key[i] : 0xFFFFFFFFu);
        hi = max(hi, key[i]);
    }
    // (fewer than k maxima above -inf, as where a mask leaves little: T is -inf)
    constexpr uint32_t NONE = 0x007FFFFFu;
    int finite = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i)
        finite += key[i] > NONE;
    if ((int)__reduce_add_sync(0xFFFFFFFFu, finite) < k)
        return -INFINITY;
    lo = max(__reduce_min_sync(0xFFFFFFFFu, lo), NONE + 1);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        int n = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i)
            n += key[i] >= mid;
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (n >= k) {
            lo = mid;
            if (n <= k + k / 4 + 2)
                break;
        } else {
            hi = mid - 1;
        }
    }
    return of_key(lo);
}

// Puts the part's k largest logits on the list, and perhaps more.  c.thread_max is written and
// c.n 0; `finder` is the warp that looks for T while warp 0 may be about the row's sums.
template <typename T>
__device__ __forceinline__ void find_top(const Part<T> &p, Candidates &c, float m, float others, int at_batch, int k,
                                         int finder)
{
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, threads = blockDim.x;
    if (warp == finder) {
        const float v = threshold(c.thread_max, lane, k);
        if (lane == 0)
            c.scratch[WARPS] = __float_as_int(v);
    }
    __syncthreads();
    const float T0 = __int_as_float(c.scratch[WARPS]);
    // the batches that reach T (a thread knows the one of its maximum; if another of its
    // batches reaches T too, all of them are read), their units among all threads
    if (m >= T0 && m > -INFINITY) {
        const int batches = (p.u1 - p.u0 - t + BATCH * threads - 1) / (BATCH * threads);
        const bool all = others >= T0 && others > -INFINITY;
        const int n = all ? batches : 1, first = atomicAdd(&c.n_chosen, n);
        for (int i = 0; i < n && first + i < CHOSEN; ++i)
            c.chosen[first + i] = (all ? i : at_batch) * THREADS + t;
    }
    __syncthreads();
    if (c.n_chosen <= CHOSEN) {
        const int items = c.n_chosen * BATCH;
        for (int i0 = t; i0 < items; i0 += 4 * threads) {
            uint4 v[4];
            int u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * threads, e = i < items ? c.chosen[i / BATCH] : 0;
                u[j] = i < items ? p.u0 + (e & (THREADS - 1)) + (e / THREADS * BATCH + i % BATCH) * threads : p.u1;
                v[j] = p.load(u[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p.each_of(v[j], u[j], [&](float x, int token) {
                    if (x >= T0 && x > -INFINITY)
                        put(c, x, token);
                });
        }
    } else if (t == 0) {
        c.n = LIST + 1;
    }
    __syncthreads();
    const int n = c.n;
    if (n > LIST) {
        float high = -INFINITY;
        for (int i = 0; i < threads; ++i)
            high = fmaxf(high, c.thread_max[i]);
        __syncthreads();
        search(p, c, T0, high, k);
        __syncthreads();
    } else if (n < k) {  // fewer than k logits above -inf
        __syncthreads();
        put_first_equal(p, c, -INFINITY, k - n);
        __syncthreads();
    }
}

// f(rank, logit, token) for the candidates of ranks below k, eight lanes to a candidate.
template <typename F>
__device__ __forceinline__ void ranked(const float *x, const int *at, int n, int k, F f)
{
    const int part = threadIdx.x & 7;
    for (int base = 0; base < n; base += blockDim.x / 8) {  // (all lanes take part in the sums)
        const int i = base + threadIdx.x / 8;
        const float v = i < n ? x[i] : 0.0f;
        const int token = i < n ? at[i] : 0;
        int rank = 0;
        for (int j = part; j < n; j += 8)
            rank += before(x[j], at[j], v, token);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
            rank += __shfl_xor_sync(0xFFFFFFFFu, rank, o);
        if (part == 0 && i < n && rank < k)
            f(rank, v, token);
    }
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(THREADS, CTAS_SM) k_token_stats(const TokenStatsArgs p, int csize, int units_cta)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N;
    __shared__ float4 part[WARPS], mine;
    __shared__ float row_m, row_ls;
    struct Lists {
        float x[MAX_TOP];
        int at[MAX_TOP];
    };
    __shared__ Candidates cand;
    __shared__ Lists own;  // a cluster's CTA: the part's k largest, ranked
    const int64_t row = blockIdx.x / csize;
    const int rank = (int)(blockIdx.x - row * csize), V = (int)p.V;
    const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5, nw = threads >> 5;
    const T *x = reinterpret_cast<const T *>(p.logits) + row * p.ld;
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int u0 = rank * units_cta;
    const Part<T> part_of = {x, V, off, u0, min(u0 + units_cta, (off + V + N - 1) / N), off ? 1 : 0, (off + V) / N};
    int64_t *ids = kTop ? p.top_ids + row * p.top : nullptr;
    float *top_lp = kTop ? p.top_lp + row * p.top : nullptr;

    const int64_t target = p.targets[row];
    if (target < 0 || target >= V) {  // an empty row, to the whole cluster
        if (rank == 0) {
            if (t == 0)
                p.lp[row] = p.lse[row] = p.entropy[row] = 0.0f;
            if (kTop)
                for (int i = t; i < p.top; i += threads) {  // (a short row has fewer threads than alternatives)
                    ids[i] = -1;
                    top_lp[i] = 0.0f;
                }
        }
        return;
    }
    float xt = 0.0f;
    if (t == 0)
        xt = E::load(x + target);
    const float c = 1.4426950408889634f / p.temperature, inv_t = p.inv_hi;
    const float2 c2 = make_float2(c, c);
    float m = -INFINITY;
    float others = -INFINITY;  // (kTop) the largest logit outside the batch of the thread's maximum
    int at_batch = 0, batch = 0;
    float2 sum = make_float2(0.0f, 0.0f), wsum = make_float2(0.0f, 0.0f);
    for (int u = u0 + t; u < part_of.u1; u += BATCH * threads, ++batch) {
        uint4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            v[i] = part_of.load(u + i * threads);
        float b = kTop ? -INFINITY : m;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            b = E::max_of(b, v[i]);
        if (kTop) {
            others = fmaxf(others, fminf(b, m));
            at_batch = b > m ? batch : at_batch;
        }
        if (b > m) {  // (m = -inf: the sums are 0, or NaN, so far)
            const float d = m == -INFINITY ? 0.0f : fmaxf((m - b) * c, LOWEST), k = ex2(d);
            wsum = __fmul2_rn(__ffma2_rn(sum, make_float2(d, d), wsum), make_float2(k, k));
            sum = __fmul2_rn(sum, make_float2(k, k));
            m = b;
        }
        // (a thread that has seen -inf only sums zeros against 0)
        const float ref = m == -INFINITY ? 0.0f : m;
        const float2 nref = make_float2(-ref, -ref);
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float2 f = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), nref), c2);
                const float2 e = make_float2(ex2(f.x), ex2(f.y));
                sum = __fadd2_rn(sum, e);
                // (a logit of -inf adds 0 x LOWEST)
                wsum = __ffma2_rn(make_float2(fmaxf(f.x, LOWEST), fmaxf(f.y, LOWEST)), e, wsum);
            }
    }
    Sums o = join({m, sum.x + sum.y, wsum.x + wsum.y}, c);
    if (lane == 0)
        part[warp] = make_float4(o.m, o.s, o.w, 0.0f);
    if (kTop) {
        cand.thread_max[t] = m;
        if (t == 0)
            cand.n = cand.n_chosen = 0;
    }
    __syncthreads();
    // the row's scalars, by lane 0 of warp 0
    auto finish = [&](const Sums &o) {
        // (not in units of log 2: the type's lowest value has a finite log probability)
        const float l2 = log2f(o.s), ls = LN2 * l2;
        const bool none = o.s == 0.0f;  // every logit is -inf
        // (NaN targets make their sum NaN; +inf - +inf too)
        p.lp[row] = none ? -INFINITY : (xt - o.m) * inv_t - ls;
        p.lse[row] = none ? -INFINITY : lse_of(o.m, ls, p.inv_hi, p.inv_lo);
        p.entropy[row] = none ? 0.0f : LN2 * (l2 - o.w / o.s);
        if (kTop) {
            row_m = o.m;
            row_ls = none ? INFINITY : ls;
        }
    };
    if (warp == 0) {
        const float4 v = lane < nw ? part[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        o = join({v.x, v.y, v.z}, c);
        if (lane == 0) {
            if (csize > 1)
                mine = make_float4(o.m, o.s, o.w, 0.0f);
            else
                finish(o);
        }
        __syncwarp();
    }
    if (kTop) {
        const int n_part = max(0, min(V, part_of.u1 * N - off) - max(0, u0 * N - off));
        const int k = min(p.top, n_part);
        if (k > 0)
            find_top(part_of, cand, m, others, at_batch, k, nw > 1 ? 1 : 0);
        if (csize > 1) {
            if (t < MAX_TOP) {
                own.x[t] = -INFINITY;
                own.at[t] = -1;
            }
            __syncthreads();
            ranked(cand.x, cand.at, min(cand.n, LIST), k, [&](int r, float v, int at) {
                own.x[r] = v;
                own.at[r] = at;
            });
        }
    }
    if (csize > 1) {
        cluster_arrive();
        cluster_wait();
        if (rank == 0) {
            if (warp == 0) {
                const float2 a = lane < csize ? ld_cluster2(reinterpret_cast<const float2 *>(&mine), lane)
                                              : make_float2(-INFINITY, 0.0f);
                const float2 b = lane < csize ? ld_cluster2(reinterpret_cast<const float2 *>(&mine) + 1, lane)
                                              : make_float2(0.0f, 0.0f);
                o = join({a.x, a.y, b.x}, c);
                if (lane == 0) {
                    finish(o);
                    cand.n = 0;
                }
                __syncwarp();
            }
            if (kTop) {  // the parts' lists, one behind the other
                __syncthreads();
                // (of which ceil(top / csize) each reach the least of those lists' elements: the rest is left out)
                const int mth = (p.top - 1) / csize;
                float least = lane < csize ? ld_cluster1(&own.x[mth], lane) : INFINITY;
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
                for (int i = t; i < csize * p.top; i += threads) {
                    const int r = i / p.top, j = i - r * p.top;
                    const float v = ld_cluster1(&own.x[j], r);
                    const int at = __float_as_int(ld_cluster1(reinterpret_cast<const float *>(&own.at[j]), r));
                    if (at >= 0 && v >= least)
                        put(cand, v, at);
                }
                __syncthreads();
            }
        }
        cluster_arrive_relaxed();  // this CTA has read the others' parts
    }
    if (kTop && rank == 0) {
        const int n = min(cand.n, LIST);
        if (n < p.top) {  // (NaN logits)
            for (int i = n + t; i < p.top; i += threads) {
                ids[i] = -1;
                top_lp[i] = NAN;
            }
        }
        const float rm = row_m, ls = row_ls;
        ranked(cand.x, cand.at, n, p.top, [&](int r, float v, int at) {
            ids[r] = at;
            top_lp[r] = v == -INFINITY && ls == ls ? -INFINITY : (v - rm) * inv_t - ls;
        });
    }
    if (csize > 1)
        cluster_wait();  // no CTA leaves while another may still read its part
}

template <typename T, bool kTop>
cudaError_t launch_stats(const TokenStatsArgs &p, cudaStream_t st)
{
    constexpr int N = Elem<T>::N;
    const int64_t units = (p.V + N - 1) / N + 1;  // one more where the rows start off a boundary
    // a row to a cluster under the loss's rule, which was fitted to that kernel (not swept for this one)
    const int64_t slots = (int64_t)CTAS_SM * device_sms();
    int csize = 1;
    while (csize < MAX_CLUSTER && 3 * p.rows * csize <= slots && units >= (int64_t)csize * 4 * THREADS)
        csize *= 2;
    const int units_cta = (int)((units + csize - 1) / csize);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * csize));
    cfg.blockDim = dim3(units_cta >= THREADS ? THREADS : (units_cta + 31) / 32 * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_token_stats<T, kTop>, p, csize, units_cta);
}

// ---------------------------------------------------------------- backward ---

constexpr int BWD_BATCH = 4, BWD_ROUNDS = 2;  // loads in flight a thread, and batches of them

// From here on an lse has too little of fp32 left for what it is subtracted from (its last rounding: 2^-17
// of a probability).
constexpr float FAR = 256.0f;

// Maximum and log2 of the sum of a row, read by one CTA, in every thread; the maximum is -inf where
// every logit is, and the sum NaN where one is a NaN or +inf.
template <typename T>
__device__ __forceinline__ float2 row_sums(const T *x, int V, int off, float c)
{
    using E = Elem<T>;
    constexpr int N = E::N;
    __shared__ float part[WARPS + 1];
    const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5, nw = threads >> 5;
    const Part<T> row = {x, V, off, 0, (off + V + N - 1) / N, off ? 1 : 0, (off + V) / N};
    float m = -INFINITY;
#pragma unroll 1
    for (int u = t; u < row.u1; u += threads)
        m = E::max_of(m, row.load(u));
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0)
        part[warp] = m;
    __syncthreads();
    for (int i = 0; i < nw; ++i)
        m = fmaxf(m, part[i]);
    __syncthreads();
    if (m == -INFINITY)
        return make_float2(m, 0.0f);
    float s = 0.0f;
#pragma unroll 1
    for (int u = t; u < row.u1; u += threads)
        row.each(u, [&](float v, int) { s += ex2((v - m) * c); });
    for (int o = 16; o; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0)
        part[warp] = s;
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < nw; ++i)
        s += part[i];
    return make_float2(m, log2f(s));
}

// A row and what its gradient takes.
template <typename T>
struct GradRow {
    using E = Elem<T>;
    static constexpr int N = E::N;
    const T *x;
    T *dx;
    int V, off, units, whole0, whole1;
    bool vec, empty;
    float lse, inv, a, b, at_target;
    int ut, jt;

    __device__ __forceinline__ GradRow(const TokenGradArgs &p, int64_t row)
    {
        V = (int)p.V;
        x = reinterpret_cast<const T *>(p.logits) + row * p.ld;
        dx = reinterpret_cast<T *>(p.dlogits) + row * p.ldd;
        off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        units = (off + V + N - 1) / N;
        whole0 = off ? 1 : 0;
        whole1 = (off + V) / N;
        // the gradient's rows share the logits' 16-byte phase: whole units leave as one store
        vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
        const int64_t target = p.targets[row];
        const float dlp = p.dlp ? p.dlp[row] : 0.0f, dH = p.dentropy ? p.dentropy[row] : 0.0f;
        lse = p.lse[row];
        empty = target < 0 || target >= V || (dlp == 0.0f && dH == 0.0f);
        inv = p.inv_hi;
        // (a row that met a NaN has lse NaN, which the maximum below would drop)
        a = lse != lse ? lse : -(dlp + (dH == 0.0f ? 0.0f : dH * p.entropy[row])) * inv;
        b = -dH * LN2 * inv;
        at_target = dlp * inv;
        const int te = (int)target + off;
        ut = te / N;
        jt = te - ut * N;
    }
    __device__ __forceinline__ void store(int u, uint4 v) const
    {
        if (vec && u >= whole0 && u < whole1)
            __stcs(reinterpret_cast<uint4 *>(dx + ((int64_t)u * N - off)), v);
        else
            store_cut(dx, u * N - off, V, v);
    }
    // Unit w's gradient, from logits less ref(...) with log2 of their sum L_hi + L_lo.
    template <typename F>
    __device__ __forceinline__ void unit(const TokenGradArgs &p, int w, const uint4 &v, float L_hi, float L_lo, F less_ref) const
    {
        const float2 a2 = make_float2(a, a), b2 = make_float2(b, b), c2 = make_float2(p.c_hi, p.c_hi),
                     cl2 = make_float2(p.c_lo, p.c_lo), nL2 = make_float2(-L_hi, -L_hi), nLl2 = make_float2(-L_lo, -L_lo);
        float2 f[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float2 e = less_ref(E::get2(v, j));
            float2 z = __fadd2_rn(__ffma2_rn(e, c2, nL2), __ffma2_rn(e, cl2, nLl2));
            // (logits of -inf: 2^LOWEST is 0)
            z = make_float2(fmaxf(z.x, LOWEST), fmaxf(z.y, LOWEST));
            f[j] = __fmul2_rn(make_float2(ex2(z.x), ex2(z.y)), __ffma2_rn(b2, z, a2));
        }
        if (w == ut) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j == jt) {
                    if (j & 1)
                        f[j / 2].y += at_target;
                    else
                        f[j / 2].x += at_target;
                }
        }
        store(w, E::pack(f));
    }
};

// A row whose lse is FAR from 0 or infinite, by one CTA.  (A call, and five CTAs an SM, so that it costs
// the others nothing: 4096 x 128256 bf16 284 us, 292 without the bound; 2048 x 1000 5.3, 5.5 as a
// part of the kernel.)
template <typename T>
__device__ __noinline__ void far_row(const TokenGradArgs &p, int64_t row)
{
    const GradRow<T> g(p, row);
    const int t = threadIdx.x, threads = blockDim.x;
    const double L = (double)g.lse * 1.4426950408889634074;
    float L_hi = (float)L, L_lo = (float)(L - L_hi);
    const float2 own = row_sums(g.x, g.V, g.off, p.c_hi);
    const float own_lse = lse_of(own.x, LN2 * own.y, p.inv_hi, p.inv_lo);
    // (an lse that is not these logits' stays what it is; without logits above -inf all is 0)
    const bool same = own_lse == g.lse || fabsf(own_lse - g.lse) <= fabsf(g.lse) * 0x1p-22f;
    const bool none = own.x == -INFINITY && g.lse == -INFINITY;
    const float nref = same && !none ? -own.x : 0.0f;
    if (same) {
        L_hi = own.y;
        L_lo = 0.0f;
    }
    const Part<T> all = {g.x, g.V, g.off, 0, g.units, g.whole0, g.whole1};
#pragma unroll 1
    for (int w = t; w < g.units; w += threads) {
        if (none)
            g.store(w, make_uint4(0, 0, 0, 0));
        else
            g.unit(p, w, all.load(w), L_hi, L_lo, [&](float2 e) { return __fadd2_rn(e, make_float2(nref, nref)); });
    }
}

// A CTA takes BWD_ROUNDS x BWD_BATCH units a thread of one row.  In units of log 2, log2 p =
// x c - L with c = log2(e) / temperature, L = lse log2(e), each a sum of two floats: one would
// put an error of 2^-24 |x c| into the exponent, some 10^-6 of a likely token's probability, and
// powers of two where a mask of -10^9 leaves a row nothing else.  There the lse itself has lost the
// sum's logarithm: of a row with such an lse the first CTA forms the sum again, and takes all of the
// row, since in place the others would overwrite what it reads.
template <typename T>
__global__ void __launch_bounds__(THREADS, 5) k_token_grad(const __grid_constant__ TokenGradArgs p, int parts)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N;
    const int64_t row = blockIdx.x / parts;
    const int partno = (int)(blockIdx.x - row * parts), t = threadIdx.x, threads = blockDim.x;
    const GradRow<T> g(p, row);
    const int span = BWD_BATCH * BWD_ROUNDS * threads;
    const int u0 = partno * span, u1 = min(u0 + span, g.units);
    if (g.empty) {
        for (int u = u0 + t; u < u1; u += threads)
            g.store(u, make_uint4(0, 0, 0, 0));
        return;
    }
    if (fabsf(g.lse) > FAR) {
        if (partno == 0)
            far_row<T>(p, row);
        return;
    }
    const double L = (double)g.lse * 1.4426950408889634074;
    const float L_hi = (float)L, L_lo = (float)(L - L_hi);
#pragma unroll 1
    for (int r = 0; r < BWD_ROUNDS; ++r) {
        const int u = u0 + t + r * BWD_BATCH * threads;
        uint4 v[BWD_BATCH];
#pragma unroll
        for (int i = 0; i < BWD_BATCH; ++i) {
            const int w = u + i * threads;
            if (w < u1)
                v[i] = w >= g.whole0 && w < g.whole1 ? ld_row(g.x + ((int64_t)w * N - g.off)) : load_cut(g.x, w * N - g.off, g.V);
        }
#pragma unroll
        for (int i = 0; i < BWD_BATCH; ++i) {
            const int w = u + i * threads;
            if (w >= u1)
                break;
            g.unit(p, w, v[i], L_hi, L_lo, [](float2 e) { return e; });
        }
    }
}

template <typename T>
cudaError_t launch_grad(const TokenGradArgs &p, cudaStream_t st)
{
    constexpr int N = Elem<T>::N;
    const int64_t units = (p.V + N - 1) / N + 1, span = (int64_t)BWD_BATCH * BWD_ROUNDS * THREADS;
    const int64_t parts = (units + span - 1) / span;
    const int threads = units < THREADS ? (int)(units + 31) / 32 * 32 : THREADS;
    return launch_pdl(k_token_grad<T>, dim3((unsigned)(p.rows * parts)), dim3(threads), 0, st, p, (int)parts);
}

}  // namespace

// 1 / temperature as the sum of two floats.
static void reciprocal(float temperature, float *hi, float *lo)
{
    *hi = 1.0f / temperature;
    *lo = (float)(1.0 / (double)temperature - (double)*hi);
}

cudaError_t launch_token_stats(const TokenStatsArgs &args, cudaStream_t st)
{
    TokenStatsArgs p = args;
    reciprocal(p.temperature, &p.inv_hi, &p.inv_lo);
    if (p.dtype == RLQ_DTYPE_F32)
        return p.top ? launch_stats<uint32_t, true>(p, st) : launch_stats<uint32_t, false>(p, st);
    return p.top ? launch_stats<uint16_t, true>(p, st) : launch_stats<uint16_t, false>(p, st);
}

cudaError_t launch_token_grad(const TokenGradArgs &args, cudaStream_t st)
{
    TokenGradArgs p = args;
    const double c = 1.4426950408889634074 / (double)p.temperature;
    p.c_hi = (float)c;
    p.c_lo = (float)(c - (double)p.c_hi);
    reciprocal(p.temperature, &p.inv_hi, &p.inv_lo);
    return p.dtype == RLQ_DTYPE_F32 ? launch_grad<uint32_t>(p, st) : launch_grad<uint16_t>(p, st);
}

}  // namespace rlq
