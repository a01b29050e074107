// Token log probabilities and the clipped policy loss over logits (sm_103a).
//
// Per row of logits x [V] with target t, z = x / temperature:
//   lp = z_t - log(sum_v exp(z_v))
//   rho = exp(lp - lp_old),  w = min(exp(lp_old - lp_behav), cap)  (1 without lp_behav)
//   pg = -w min(rho A, clip(rho, 1 - eps_lo, hi) A),  hi = clip_hi[row] or 1 + eps_hi
//   kl = beta (exp(d) - 1 - d),  d = lp_ref - lp
//   loss = weight (pg + kl)
//   dloss/dlp = weight (-w A rho [the unclipped branch is the minimum] - beta (exp(d) - 1))
//   dlogits_v = dloss/dlp (1[v = t] - softmax(z)_v) / temperature
//
// Bound by memory: the logits are read once and the gradient written once.  Without a
// gradient a row is streamed (k_token_rows).  With one it is held on chip by one CTA, or
// by a cluster of 2, 4 or 8 for long rows (k_policy_grad), persistent CTAs: one warp copies
// the next rows to shared memory (bulk copies), another joins the reducing warps'
// (maximum, sum) pairs of a row across the cluster and publishes the row's factors, while
// those warps already reduce the next row; they write a row's gradient after that.  So a
// row's chain of latencies (cluster barrier, remote reads, logarithm and exponentials)
// lies beside the work on its neighbours.  The gradient may overwrite the logits: a row
// is read whole before any of it is written.
#include <cuda_runtime.h>

#include <mutex>

#include "rlq_elem.cuh"
#include "rlq_internal.h"
#include "rlq_tc.cuh"

namespace rlq {
namespace {

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {  // bf16
    static constexpr int N = 8;  // elements per 16 bytes
    static __device__ __forceinline__ float2 get2(const uint4 &v, int j)  // elements 2j, 2j + 1
    {
        const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
        return make_float2(bf_lo(w), bf_hi(w));
    }
    // maximum of m and the unit's elements; NaN is passed over
    static __device__ __forceinline__ float max_of(float m, const uint4 &v)
    {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fmaxf(m, fmaxf(bf_lo(a), bf_hi(a)));
    }
    static __device__ __forceinline__ float load(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[4])
    {
        return make_uint4(pack_bf16x2(f[0]), pack_bf16x2(f[1]), pack_bf16x2(f[2]), pack_bf16x2(f[3]));
    }
};
template <>
struct Elem<uint32_t> {  // fp32
    static constexpr int N = 4;
    static __device__ __forceinline__ float2 get2(const uint4 &v, int j)
    {
        return j == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                      : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ float max_of(float m, const uint4 &v)
    {
        return fmaxf(fmaxf(m, __uint_as_float(v.x)),
                     fmaxf(fmaxf(__uint_as_float(v.y), __uint_as_float(v.z)), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ float load(const uint32_t *p) { return __uint_as_float(*p); }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[2])
    {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                          __float_as_uint(f[1].y));
    }
};

// 2^x, results below 2^-126 flushed to zero (one instruction).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Global -> shared bulk copy of `bytes` (a multiple of 16, both addresses 16-byte
// aligned), completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ float2 ld_cluster2(uint32_t a, uint32_t rank)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(cluster_addr(a, rank))
                 : "memory");
    return v;
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// An arrival that orders nothing: it does not wait for the thread's own stores.
__device__ __forceinline__ void cluster_arrive_relaxed()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct RowScalars {
    float lp, lse, loss, dlp;
};

// A row's inputs of the loss, loaded ahead of their use.
struct RowInputs {
    float old, adv, weight, behav, ref, hi;
};

__device__ __forceinline__ RowInputs row_inputs(const PolicyLossArgs &p, int64_t row)
{
    RowInputs in = {};
    if (p.adv) {
        in.old = p.lp_old[row];
        in.adv = p.adv[row];
        in.weight = p.weight[row];
        in.behav = p.lp_behav ? p.lp_behav[row] : 0.0f;
        in.ref = p.lp_ref ? p.lp_ref[row] : 0.0f;
        in.hi = p.clip_hi ? p.clip_hi[row] : 1.0f + p.eps_hi;
    }
    return in;
}

// (maximum, sum of 2^((x - maximum) c)) pairs of a warp's lanes, joined in every lane.  A
// pair of -inf only has the sum 0; one of NaN has no maximum but a NaN sum.
__device__ __forceinline__ float2 join_pairs(float2 v, float c)
{
    float m = v.x;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float s = v.y == 0.0f ? 0.0f : v.y * ex2((v.x - m) * c);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return make_float2(m, s);
}

// The row's loss and its derivative, from the row's maximum (m, in logits), the sum S
// of 2^((x - m) c) and the target's logit.
__device__ __noinline__ RowScalars row_scalars(const PolicyLossArgs &p, const RowInputs in, float m, float S,
                                                float xt, float c)
{
    RowScalars o;
    constexpr float LN2 = 0.6931471805599453f;
    if (S == 0.0f) {  // every logit is -inf: an empty row
        o.lp = o.lse = -INFINITY;
        o.loss = o.dlp = 0.0f;
        return o;
    }
    o.lp = LN2 * ((xt - m) * c - log2f(S));
    o.lse = fmaf(m, c * LN2, LN2 * log2f(S));
    o.loss = o.dlp = 0.0f;
    if (!p.adv)
        return o;
    const float rho = expf(o.lp - in.old);
    const float isw = p.lp_behav ? fminf(expf(in.old - in.behav), p.tis_cap) : 1.0f;
    const float plain = rho * in.adv, clipped = fminf(fmaxf(rho, 1.0f - p.eps_lo), in.hi) * in.adv;
    float loss = -isw * fminf(plain, clipped);
    float dlp = plain <= clipped ? -isw * plain : 0.0f;
    if (p.lp_ref) {
        const float d = in.ref - o.lp, e = expm1f(d);
        loss = fmaf(p.kl_beta, e - d, loss);
        dlp = fmaf(-p.kl_beta, e, dlp);
    }
    o.loss = in.weight * loss;
    o.dlp = in.weight * dlp;
    return o;
}

// The elements of the unit at e0 .. of a row of V, those outside the row as -inf.
template <typename T>
__device__ __forceinline__ void load_edge(const T *x, int e0, int V, T (&raw)[Elem<T>::N])
{
#pragma unroll
    for (int j = 0; j < Elem<T>::N; ++j)
        raw[j] = e0 + j >= 0 && e0 + j < V ? x[e0 + j] : (T)(sizeof(T) == 2 ? 0xFF80u : 0xFF800000u);
}

template <typename T>
__device__ __forceinline__ uint4 join_edge(const T (&raw)[Elem<T>::N])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = sizeof(T) == 2 ? (uint32_t)raw[(2 * j) % Elem<T>::N] | ((uint32_t)raw[(2 * j + 1) % Elem<T>::N] << 16)
                              : (uint32_t)raw[j];
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// (both out of line: a row has at most one such unit at each end)
template <typename T>
__device__ __noinline__ uint4 load_cut(const T *x, int e0, int V)
{
    T raw[Elem<T>::N];
    load_edge(x, e0, V, raw);
    return join_edge<T>(raw);
}

template <typename T>
__device__ __noinline__ void store_edge(T *dx, int e0, int V, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < Elem<T>::N; ++j)
        if (e0 + j >= 0 && e0 + j < V)
            dx[e0 + j] = sizeof(T) == 2 ? (T)(w[j / 2] >> (16 * (j & 1))) : (T)w[j & 3];
}

// Log probabilities, or the loss without its gradient: nothing of the row is needed
// again, so a CTA streams its part of it once, keeping a running maximum and sum a
// thread, 8 loads of 16 bytes in flight.  A row is one CTA's, or a cluster's of 2, 4 or 8
// where there are few rows; unit and rank as below.
template <typename T>
__global__ void __launch_bounds__(256, 4) k_token_rows(const PolicyLossArgs p, int csize, int units_cta)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N, BATCH = 8;
    constexpr uint32_t NINF = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    __shared__ float2 pairs[8], mine;
    const int64_t row = blockIdx.x / csize;
    const int rank = (int)(blockIdx.x - row * csize), V = (int)p.V;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x >> 5;
    const T *x = reinterpret_cast<const T *>(p.logits) + row * p.ld;
    const int64_t target = p.targets[row];
    if (target < 0 || target >= V || (p.weight && p.weight[row] == 0.0f)) {  // an empty row, to the whole cluster
        if (rank == 0 && t == 0) {
            p.lp[row] = 0.0f;
            if (p.lse)
                p.lse[row] = 0.0f;
            if (p.loss)
                p.loss[row] = 0.0f;
        }
        return;
    }
    float xt = 0.0f;
    RowInputs in = {};
    if (rank == 0 && warp == 0) {
        xt = E::load(x + target);
        in = row_inputs(p, row);
    }
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int u0 = rank * units_cta, u1 = min(u0 + units_cta, (off + V + N - 1) / N);
    const int whole0 = off ? 1 : 0, whole1 = (off + V) / N;  // units that the row's ends do not cut
    const float c = 1.4426950408889634f / p.temperature;
    const float2 c2 = make_float2(c, c);
    float m = -INFINITY;
    float2 sum = make_float2(0.0f, 0.0f);
    for (int u = u0 + t; u < u1; u += BATCH * blockDim.x) {
        uint4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int w = u + i * (int)blockDim.x;
            v[i] = make_uint4(NINF, NINF, NINF, NINF);
            if (w < u1 && w >= whole0 && w < whole1)
                v[i] = ld_stream(reinterpret_cast<const uint16_t *>(x + ((int64_t)w * N - off)));
            else if (w < u1)
                v[i] = load_cut(x, w * N - off, V);
        }
        float b = m;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            b = E::max_of(b, v[i]);
        // (a thread that has seen -inf only sums zeros against 0)
        const float ref = b == -INFINITY ? 0.0f : b;
        if (b > m) {
            const float k = m == -INFINITY ? (sum.x + sum.y == 0.0f ? 0.0f : 1.0f) : ex2((m - b) * c);
            sum = __fmul2_rn(sum, make_float2(k, k));
            m = b;
        }
        const float2 nref = make_float2(-ref, -ref);
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float2 f = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), nref), c2);
                sum = __fadd2_rn(sum, make_float2(ex2(f.x), ex2(f.y)));
            }
    }
    float2 o = join_pairs(make_float2(m, sum.x + sum.y), c);
    if (lane == 0)
        pairs[warp] = o;
    __syncthreads();
    if (warp == 0) {
        o = join_pairs(lane < nw ? pairs[lane] : make_float2(-INFINITY, 0.0f), c);
        if (lane == 0)
            mine = o;
    }
    if (csize > 1) {
        __syncwarp();
        cluster_sync();
        if (rank == 0 && warp == 0)
            o = join_pairs(lane < csize ? ld_cluster2(smem_u32(&mine), lane) : make_float2(-INFINITY, 0.0f), c);
        __syncwarp();
    }
    if (rank == 0 && warp == 0) {
        const RowScalars r = row_scalars(p, in, o.x, o.y, xt, c);
        if (lane == 0) {
            p.lp[row] = r.lp;
            if (p.lse)
                p.lse[row] = r.lse;
            if (p.loss)
                p.loss[row] = r.loss;
        }
    }
    if (csize > 1)
        cluster_sync();  // no CTA leaves while another may still read its pair
}

constexpr int MAX_BUFS = 3;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_WARPS = 16;  // that reduce, beside the joining and the copying warp

struct RowsPlan {
    int csize;      // CTAs of a cluster (of a row)
    int units_cta;  // 16-byte units of a row per CTA
    int bufs;       // rows held in shared memory
    uint64_t timeout_ns;
};

// A persistent cluster takes rows cluster, cluster + clusters, ...  Units are a row's
// 16-byte pieces on 16-byte boundaries: unit u covers elements u N - off .. + N - 1, off
// being the elements by which the row starts past a boundary.  The CTA of rank c takes
// units c units_cta .. (c + 1) units_cta - 1, thread t of its reducing warps units t,
// t + threads, ... of those.  Whole units come by bulk copy; a unit that the row's start or
// end cuts is put into shared memory by the copying warp, the missing elements as -inf.
// Empty rows are not copied, so buffers and phases go by the count of live rows.
//
// Per live row L, the reducing warps reduce L, then write the gradient of L - 1 (with a
// single buffer: of L); the joining warp joins L and publishes its factors; the copying
// warp copies the row bufs - 1 (or 1) ahead, whose buffer's last row was at most L - 1
// (or L) and is released by the reducing warps without its doing.  All warps of a
// cluster meet in one hardware barrier per live row, behind which L's pairs are there:
// a CTA's reducing warps hand their pairs to its joining warp (an mbarrier), whose
// arrival alone releases them to the cluster.  (A releasing arrival of the reducing
// warps waits for the gradient's stores at every row: 479 us against 439 for 4096 rows
// of 128256.)
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 320 ? 2 : 1)
    k_policy_grad(const PolicyLossArgs p, const RowsPlan plan)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N;
    extern __shared__ __align__(128) uint8_t data[];  // [bufs][units_cta] units
    // by the parity of the live row: this CTA's warps' pairs, the row's factors
    __shared__ __align__(16) float2 pairs[2][MAX_WARPS];
    __shared__ float4 coef[2];  // -dz / sum, the maximum, dz
    // Barriers: a buffer's row is there (one arrival by the copy, one by the cut units),
    // a buffer is free (each reducing warp), this CTA's pairs are there, the factors are
    __shared__ __align__(8) uint64_t full_bars[MAX_BUFS], empty_bars[MAX_BUFS], pair_bars[2], coef_bars[2];
    __shared__ uint32_t abort_word;
    volatile uint32_t *abort_flag = &abort_word;
    const int csize = plan.csize, cap = plan.units_cta, bufs = plan.bufs, lag = bufs > 1 ? 1 : 0;
    const int64_t clusters = gridDim.x / csize, first = blockIdx.x / csize;
    const int rank = (int)(blockIdx.x - first * csize);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = (blockDim.x >> 5) - 2;
    const int V = (int)p.V, u0 = rank * cap;
    const T *logits = reinterpret_cast<const T *>(p.logits);
    const float c = 1.4426950408889634f / p.temperature;
    const float2 c2 = make_float2(c, c);

    auto live_row = [&](int64_t target, float weight) { return target >= 0 && target < V && weight != 0.0f; };
    auto offset = [&](const T *x) { return (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)); };
    // A wait that runs out is reported by rlq_check; its warp goes on, without waiting any
    // more, so that the cluster's CTAs end together.
    auto wait = [&](uint64_t *bar, int phase) {
        if (!*abort_flag)
            mbar_wait(smem_u32(bar), (uint32_t)phase & 1u, abort_flag, plan.timeout_ns, SITE_LOSS_ROW);
        __syncwarp();
    };

    if (t == 0) {
        for (int b = 0; b < bufs; ++b) {
            mbar_init(smem_u32(&full_bars[b]), 2);
            mbar_init(smem_u32(&empty_bars[b]), nw);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&pair_bars[b]), nw);
            mbar_init(smem_u32(&coef_bars[b]), 1);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();

    int64_t target = p.targets[first];
    float weight = p.weight ? p.weight[first] : 1.0f;
    int nlive = 0;  // live rows so far
    if (warp == nw + 1) {
        // -------------------------------------------------- copying warp ---
        int64_t ahead = first;
        int ahead_live = 0;
        // copies this CTA's part of row `ahead` into its buffer, if it is live
        auto refill = [&](int64_t tg, float w) {
            if (ahead >= p.rows || !live_row(tg, w))
                return;
            const int buf = ahead_live % bufs, use = ahead_live / bufs;
            if (use > 0)
                wait(&empty_bars[buf], use - 1);
            const T *x = logits + ahead * p.ld;
            const int off = offset(x), last = (off + V) / N;  // the first unit not wholly before the row's end
            uint4 *dst = reinterpret_cast<uint4 *>(data) + buf * cap;
            if (lane == 0) {
                const int a = max(u0, off ? 1 : 0), b = min(u0 + cap, last);
                const uint32_t bytes = b > a ? (uint32_t)(b - a) * 16u : 0u;
                mbar_arrive_expect_tx(smem_u32(&full_bars[buf]), bytes);
                if (bytes)
                    bulk_load(smem_u32(dst + a - u0), x + ((int64_t)a * N - off), bytes, smem_u32(&full_bars[buf]));
            }
            // cut units: the row's first (lane 0) and last (lane 1; lane 0's if it is the same)
            int u = -1;
            if (lane == 0 && off != 0)
                u = 0;
            else if (lane == 1 && (off + V) % N != 0 && !(off != 0 && last == 0))
                u = last;
            if (u >= u0 && u < u0 + cap) {
                T raw[N];
                load_edge(x, u * N - off, V, raw);
                dst[u - u0] = join_edge<T>(raw);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&full_bars[buf]));
            ++ahead_live;
        };
        for (int b = 0; b < bufs - lag && ahead < p.rows; ++b, ahead += clusters)
            refill(p.targets[ahead], p.weight ? p.weight[ahead] : 1.0f);
        for (int64_t row = first; row < p.rows; row += clusters, ahead += clusters) {
            const bool live = live_row(target, weight);
            // what the next iteration and the refill need, loaded early
            if (row + clusters < p.rows) {
                target = p.targets[row + clusters];
                weight = p.weight ? p.weight[row + clusters] : 1.0f;
            }
            int64_t ahead_target = -1;
            float ahead_weight = 1.0f;
            if (ahead < p.rows) {
                ahead_target = p.targets[ahead];
                ahead_weight = p.weight ? p.weight[ahead] : 1.0f;
            }
            if (live && csize > 1) {
                cluster_arrive_relaxed();
                cluster_wait();
            }
            refill(ahead_target, ahead_weight);
        }
    } else if (warp == nw) {
        // -------------------------------------------------- joining warp ---
        // A row's inputs are loaded while the row before is joined.
        float xt = 0.0f;
        RowInputs in = {};
        auto load_inputs = [&](int64_t row) {
            if (row >= p.rows || !live_row(target, weight))
                return;
            xt = E::load(logits + row * p.ld + target);
            in = row_inputs(p, row);
        };
        load_inputs(first);
        for (int64_t row = first; row < p.rows; row += clusters) {
            const bool live = live_row(target, weight);
            if (row + clusters < p.rows) {
                target = p.targets[row + clusters];
                weight = p.weight ? p.weight[row + clusters] : 1.0f;
            }
            if (!live) {
                if (rank == 0 && lane == 0) {
                    p.lp[row] = 0.0f;
                    if (p.lse)
                        p.lse[row] = 0.0f;
                    if (p.loss)
                        p.loss[row] = 0.0f;
                }
                load_inputs(row + clusters);
                continue;
            }
            const int par = nlive & 1;
            // (the vote has the arrival, and so any write to the row, wait for the load of xt)
            const float x_t = xt;
            const RowInputs now = in;
            const bool nan_target = __any_sync(0xFFFFFFFFu, x_t != x_t);
            wait(&pair_bars[par], nlive >> 1);
            if (csize > 1) {
                cluster_arrive();
                cluster_wait();
            }
            float2 o[MAX_CLUSTER * MAX_WARPS / 32];
            float gm = -INFINITY, G = 0.0f;
#pragma unroll
            for (int k = 0; k < MAX_CLUSTER * MAX_WARPS / 32; ++k) {
                // entry e: warp e % 16 of rank e / 16 (the same order in every CTA)
                const int e = lane + 32 * k, r = e / MAX_WARPS, w = e % MAX_WARPS;
                o[k] = make_float2(-INFINITY, 0.0f);
                if (r < csize && w < nw)
                    o[k] = csize > 1 ? ld_cluster2(smem_u32(&pairs[par][w]), r) : pairs[par][w];
            }
            load_inputs(row + clusters);
#pragma unroll
            for (int k = 0; k < MAX_CLUSTER * MAX_WARPS / 32; ++k)
                gm = fmaxf(gm, o[k].x);
#pragma unroll
            for (int k = 16; k; k >>= 1)
                gm = fmaxf(gm, __shfl_xor_sync(0xFFFFFFFFu, gm, k));
            // (a part of -inf only has the sum 0; one of NaN has no maximum but a NaN sum)
#pragma unroll
            for (int k = 0; k < MAX_CLUSTER * MAX_WARPS / 32; ++k)
                G += o[k].y == 0.0f ? 0.0f : o[k].y * ex2((o[k].x - gm) * c);
#pragma unroll
            for (int k = 16; k; k >>= 1)
                G += __shfl_xor_sync(0xFFFFFFFFu, G, k);
            if (nan_target)
                G = x_t;
            const RowScalars r = row_scalars(p, now, gm, G, x_t, c);
            if (lane == 0) {
                const float dz = r.dlp / p.temperature;
                // -dz * softmax; an empty row's probabilities are 0
                coef[par] = make_float4(G == 0.0f ? 0.0f : -dz / G, gm == -INFINITY ? 0.0f : gm, dz, 0.0f);
                mbar_arrive(smem_u32(&coef_bars[par]));
                if (rank == 0) {
                    p.lp[row] = r.lp;
                    if (p.lse)
                        p.lse[row] = r.lse;
                    if (p.loss)
                        p.loss[row] = r.loss;
                }
            }
            __syncwarp();
            ++nlive;
        }
    } else {
        // ---------------------------------------------- reducing warps ---
        const int threads = nw * 32;
        // The gradient of live row number `n` (row `row`, target `tgt`), behind its factors;
        // then the row's buffer is free.
        auto finish = [&](int n, int64_t row, int64_t tgt) {
            wait(&coef_bars[n & 1], n >> 1);
            const int buf = n % bufs;
            T *dx = reinterpret_cast<T *>(p.dlogits) + row * p.ldd;
            const T *x = logits + row * p.ld;
            const int off = offset(x), units = min(cap, (off + V + N - 1) / N - u0);
            // rows that share the logits' 16-byte phase: whole units leave as one store
            const bool vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
            const uint4 *src = reinterpret_cast<const uint4 *>(data) + buf * cap;
            const float4 k4 = coef[n & 1];
            const float2 f2 = make_float2(k4.x, k4.x), ng2 = make_float2(-k4.y, -k4.y);
            const int te = (int)tgt + off, ut = te / N - u0, jt = te % N;
            const int lo = vec ? (off && u0 == 0 ? 1 : 0) : cap, hi = vec ? (off + V) / N - u0 : 0;
            T *dst = dx + ((int64_t)u0 * N - off);
#pragma unroll 4
            for (int u = t; u < units; u += threads) {
                const uint4 v = src[u];
                float2 f[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 z = __fmul2_rn(__fadd2_rn(E::get2(v, j), ng2), c2);
                    f[j] = __fmul2_rn(make_float2(ex2(z.x), ex2(z.y)), f2);
                }
                if (u == ut) {
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j == jt) {
                            if (j & 1)
                                f[j / 2].y += k4.z;
                            else
                                f[j / 2].x += k4.z;
                        }
                }
                if (u >= lo && u < hi)
                    *reinterpret_cast<uint4 *>(dst + u * N) = E::pack(f);
                else
                    store_edge(dx, (u0 + u) * N - off, V, E::pack(f));
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&empty_bars[buf]));
        };
        int64_t last_row = -1, last_target = 0;  // the live row whose gradient is due
        for (int64_t row = first; row < p.rows; row += clusters) {
            const int64_t tgt = target;
            const bool live = live_row(target, weight);
            if (row + clusters < p.rows) {
                target = p.targets[row + clusters];
                weight = p.weight ? p.weight[row + clusters] : 1.0f;
            }
            const T *x = logits + row * p.ld;
            const int off = offset(x), units = min(cap, (off + V + N - 1) / N - u0);
            if (!live) {
                T *dx = reinterpret_cast<T *>(p.dlogits) + row * p.ldd;
                const bool vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
                for (int u = t; u < units; u += threads) {
                    const int e0 = (u0 + u) * N - off;
                    if (vec && e0 >= 0 && e0 + N <= V)
                        *reinterpret_cast<uint4 *>(dx + e0) = make_uint4(0, 0, 0, 0);
                    else
                        store_edge(dx, e0, V, make_uint4(0, 0, 0, 0));
                }
                continue;
            }
            const int buf = nlive % bufs, par = nlive & 1;
            wait(&full_bars[buf], nlive / bufs);
            const uint4 *src = reinterpret_cast<const uint4 *>(data) + buf * cap;
            float m = -INFINITY;
#pragma unroll 4
            for (int u = t; u < units; u += threads)
                m = E::max_of(m, src[u]);
            // a part that is all -inf sums zeros against any finite maximum
            const float mm = m == -INFINITY ? 0.0f : m;
            const float2 nm2 = make_float2(-mm, -mm);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 4
            for (int u = t; u < units; u += threads) {
                const uint4 v = src[u];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 f = __fmul2_rn(__fadd2_rn(E::get2(v, j), nm2), c2);
                    sum = __fadd2_rn(sum, make_float2(ex2(f.x), ex2(f.y)));
                }
            }
            const float2 pair = join_pairs(make_float2(m, sum.x + sum.y), c);
            // (pairs of this parity were joined before the factors that finish() of the row
            // two before waited for, in a cluster before the barrier of the row before)
            if (lane == 0)
                pairs[par][warp] = pair;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&pair_bars[par]));
            __syncwarp();
            if (csize > 1)
                cluster_arrive_relaxed();
            if (!lag)
                finish(nlive, row, tgt);
            else if (last_row >= 0)
                finish(nlive - 1, last_row, last_target);
            last_row = row;
            last_target = tgt;
            if (csize > 1)
                cluster_wait();
            ++nlive;
        }
        if (lag && last_row >= 0)
            finish(nlive - 1, last_row, last_target);
    }
    if (*abort_flag) {  // copies may still be in flight: they have some time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull)
            __nanosleep(1000);
    }
    if (csize > 1)
        cluster_sync();  // no CTA leaves while another may still read its pairs
}

// CTAs (in whole clusters) that are resident at once, looked up once per launch shape.
template <typename Kernel>
cudaError_t resident_ctas(Kernel kernel, const cudaLaunchConfig_t &cfg, int csize, int *ctas)
{
    struct Known {
        const void *kernel;
        int dev, csize;
        size_t smem;
        unsigned threads;
        int ctas;
    };
    static Known known[64];
    static int count = 0;
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const void *id = reinterpret_cast<const void *>(kernel);
    std::lock_guard<std::mutex> g(mu);
    for (int i = 0; i < count && i < 64; ++i)
        if (known[i].kernel == id && known[i].dev == dev && known[i].csize == csize &&
            known[i].smem == cfg.dynamicSmemBytes && known[i].threads == cfg.blockDim.x) {
            *ctas = known[i].ctas;
            return cudaSuccess;
        }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 4096);
    if (e != cudaSuccess)
        return e;
    int n = 0;
    if (csize == 1) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, (int)cfg.blockDim.x, cfg.dynamicSmemBytes);
        n *= device_sms();
    } else {
        cudaLaunchConfig_t q = cfg;
        q.gridDim = dim3((unsigned)(csize * device_sms()));
        q.attrs = cfg.attrs + 1;  // the cluster's shape alone
        q.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        n *= csize;
    }
    if (e != cudaSuccess)
        return e;
    if (n < csize)
        return cudaErrorLaunchOutOfResources;
    known[count % 64] = {id, dev, csize, cfg.dynamicSmemBytes, cfg.blockDim.x, n};
    ++count;
    *ctas = n;
    return cudaSuccess;
}

template <typename T, int kThreads>
cudaError_t launch_rows(const PolicyLossArgs &p, const RowsPlan &plan, int threads, cudaStream_t st)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = plan.csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)plan.bufs * plan.units_cta * 16;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = plan.csize > 1 ? 2 : 1;
    auto kernel = k_policy_grad<T, kThreads>;
    int ctas = 0;
    const cudaError_t e = resident_ctas(kernel, cfg, plan.csize, &ctas);
    if (e != cudaSuccess)
        return e;
    const int64_t want = p.rows * plan.csize;
    cfg.gridDim = dim3((unsigned)(want < ctas ? want : ctas));
    return cudaLaunchKernelEx(&cfg, kernel, p, plan);
}

constexpr int64_t SMEM_CTA = 220 * 1024;  // of 227 KB, beside the pairs and what the system keeps

template <typename T>
cudaError_t launch_forward(const PolicyLossArgs &p, int64_t units, cudaStream_t st)
{
    // rows over clusters until every SM has four CTAs, while a thread keeps two units
    int csize = 1;
    while (csize < MAX_CLUSTER && p.rows * csize < 4 * device_sms() && units >= (int64_t)csize * 2 * 512)
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
    cfg.blockDim = dim3(units_cta >= 256 ? 256 : (units_cta + 31) / 32 * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_token_rows<T>, p, csize, units_cta);
}

template <typename T>
cudaError_t launch_typed(const PolicyLossArgs &p, cudaStream_t st)
{
    constexpr int N = Elem<T>::N;
    const int64_t units = (p.V + N - 1) / N + 1;  // one more where the rows start off a boundary
    if (!p.dlogits)
        return launch_forward<T>(p, units, st);
    // a row in one CTA of at most 32 KB, else in the smallest cluster whose CTAs hold
    // that, else in a cluster of 8 with more per CTA
    int csize = 1;
    while (csize < MAX_CLUSTER && units > (int64_t)csize * 2048)
        csize *= 2;
    RowsPlan plan;
    plan.csize = csize;
    plan.units_cta = (int)((units + csize - 1) / csize);
    plan.timeout_ns = wait_limit_ns();
    const int64_t row = (int64_t)plan.units_cta * 16;
    // two CTAs per SM where that leaves each three rows, else one
    const int64_t room = 6 * row <= SMEM_CTA ? SMEM_CTA / 2 : SMEM_CTA;
    plan.bufs = (int)(room / row < MAX_BUFS ? room / row : MAX_BUFS);
    // the reducing warps, the joining and the copying one
    if (plan.units_cta > 2304)
        return launch_rows<T, 576>(p, plan, 576, st);
    const int threads = plan.units_cta >= 256 ? 256 : (plan.units_cta + 31) / 32 * 32;
    return launch_rows<T, 320>(p, plan, threads + 64, st);
}

}  // namespace

int64_t policy_max_vocab(int dtype) { return (int64_t)8 * 512 * 16 * (dtype == RLQ_DTYPE_F32 ? 4 : 8) - 8; }

cudaError_t take_loss_error_word(cudaStream_t st, unsigned long long *word) { return take_error_word(st, word); }

cudaError_t launch_policy_rows(const PolicyLossArgs &p, cudaStream_t st)
{
    return p.dtype == RLQ_DTYPE_F32 ? launch_typed<uint32_t>(p, st) : launch_typed<uint16_t>(p, st);
}

}  // namespace rlq
