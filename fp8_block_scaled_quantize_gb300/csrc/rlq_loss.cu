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
// Bound by memory: the logits are read once and the gradient written once.  A row is
// held on chip by one CTA, or by a cluster of 2, 4 or 8 for long rows: a persistent
// cluster copies its next rows to shared memory (bulk copies, up to three rows ahead)
// while it works on one.  A thread takes its part of the row into registers, its
// maximum and the sum of its exponentials; behind one cluster barrier per row the first
// warp of each CTA joins all warps' (maximum, sum) pairs, read from the CTAs' shared
// memory, and publishes the row's factors, and every warp writes its part of the
// gradient.  The gradient may overwrite the logits: a row is read whole before any of
// it is written.
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
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct RowScalars {
    float lp, lse, loss, dlp;
};

// A row's inputs of the loss, loaded ahead of their use.
struct RowInputs {
    float old, adv, weight, behav, ref, hi;
};

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

// (out of line: a row has at most one such unit at each end)
template <typename T>
__device__ __noinline__ void store_edge(T *dx, int e0, int V, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < Elem<T>::N; ++j)
        if (e0 + j >= 0 && e0 + j < V)
            dx[e0 + j] = sizeof(T) == 2 ? (T)(w[j / 2] >> (16 * (j & 1))) : (T)w[j & 3];
}

constexpr int MAX_BUFS = 3;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_WARPS = 16;

struct RowsPlan {
    int csize;      // CTAs of a cluster (of a row)
    int units_cta;  // 16-byte units of a row per CTA
    int bufs;       // rows held in shared memory
    uint64_t timeout_ns;
};

// A persistent cluster takes rows cluster, cluster + clusters, ...  Units are a row's
// 16-byte pieces on 16-byte boundaries: unit u covers elements u N - off .. + N - 1, off
// being the elements by which the row starts past a boundary.  The CTA of rank c takes
// units c units_cta .. (c + 1) units_cta - 1, thread t of it units t + i * blockDim.x, i < NV.
// Whole units come by bulk copy; a unit that the row's start or end cuts is put into
// shared memory by a thread of the last warp, the missing elements as -inf.  Empty rows
// are not copied, so buffers and their phases go by the count of live rows.
template <typename T, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 256 ? 2 : 1)
    k_policy_rows(const PolicyLossArgs p, const RowsPlan plan)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N;
    extern __shared__ __align__(128) uint8_t data[];  // [bufs][units_cta] units
    // by the parity of the live row: this CTA's warps' pairs, the row's factors
    __shared__ __align__(16) float2 pairs[2][MAX_WARPS];
    // Barriers: a buffer's row is there (one arrival by its copier, one by the warp that
    // fills in cut units); the row's factors are there
    __shared__ __align__(8) uint64_t bars[MAX_BUFS], coef_bars[2];
    __shared__ float4 coef[2];  // -dz / sum, the maximum, dz
    __shared__ uint32_t abort_word;
    volatile uint32_t *abort_flag = &abort_word;
    const int csize = plan.csize, cap = plan.units_cta, bufs = plan.bufs;
    const int64_t clusters = gridDim.x / csize, first = blockIdx.x / csize;
    const int rank = (int)(blockIdx.x - first * csize);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x >> 5;
    const int V = (int)p.V, u0 = rank * cap;
    const uint32_t data0 = smem_u32(data);
    const T *logits = reinterpret_cast<const T *>(p.logits);
    const float c = 1.4426950408889634f / p.temperature;
    const float2 c2 = make_float2(c, c);

    auto live_row = [&](int64_t target, float weight) { return target >= 0 && target < V && weight != 0.0f; };
    auto offset = [&](const T *x) { return (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)); };
    // copies this CTA's whole units of a row (one thread)
    auto issue = [&](int64_t row, int buf) {
        const T *x = logits + row * p.ld;
        const int off = offset(x);
        const int a = max(u0, off ? 1 : 0), b = min(u0 + cap, (off + V) / N);
        const uint32_t bytes = b > a ? (uint32_t)(b - a) * 16u : 0u;
        mbar_arrive_expect_tx(smem_u32(&bars[buf]), bytes);
        if (bytes)
            bulk_load(data0 + (uint32_t)(buf * cap + a - u0) * 16u, x + ((int64_t)a * N - off), bytes,
                      smem_u32(&bars[buf]));
    };
    // the unit that this lane of the last warp fills in: the row's first where it is cut
    // (lane 0), its last where it is cut (lane 1; the same unit of a very short row is
    // lane 0's); -1: none here
    auto edge_unit = [&](const T *x) {
        const int off = offset(x), last = (off + V) / N;  // the first unit not wholly before the row's end
        const bool cut0 = off != 0, cut1 = (off + V) % N != 0;
        int u = -1;
        if (lane == 0 && cut0)
            u = 0;
        else if (lane == 1 && cut1 && !(cut0 && last == 0))
            u = last;
        return u >= u0 && u < u0 + cap ? u : -1;
    };

    if (t == 0) {
        for (int b = 0; b < bufs; ++b)
            mbar_init(smem_u32(&bars[b]), 2);
        for (int b = 0; b < 2; ++b)
            mbar_init(smem_u32(&coef_bars[b]), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    // The rows ahead: row index, and the count of live rows in front of it.
    int64_t ahead = first;
    int ahead_live = 0;
    for (int b = 0; b < bufs && ahead < p.rows; ++b, ahead += clusters) {
        if (!live_row(p.targets[ahead], p.weight ? p.weight[ahead] : 1.0f))
            continue;
        if (t == 0)
            issue(ahead, ahead_live % bufs);
        if (warp == nw - 1) {
            const T *x = logits + ahead * p.ld;
            const int u = edge_unit(x);
            if (u >= 0) {
                T raw[N];
                load_edge(x, u * N - offset(x), V, raw);
                reinterpret_cast<uint4 *>(data)[(ahead_live % bufs) * cap + u - u0] = join_edge<T>(raw);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bars[ahead_live % bufs]));
        }
        ++ahead_live;
    }

    int64_t target = 0;
    float weight = 0.0f;
    if (first < p.rows) {
        target = p.targets[first];
        weight = p.weight ? p.weight[first] : 1.0f;
    }
    int nlive = 0;  // live rows so far
    for (int64_t row = first; row < p.rows; row += clusters, ahead += clusters) {
        const T *x = logits + row * p.ld;
        T *dx = p.dlogits ? reinterpret_cast<T *>(p.dlogits) + row * p.ldd : nullptr;
        const int off = offset(x), u1 = min(u0 + cap, (off + V + N - 1) / N);
        // the gradient's rows share the logits' 16-byte phase: whole units leave as one store
        const bool vec_out = dx && ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
        auto store = [&](int u, const float2(&f)[N / 2]) {
            const int e0 = u * N - off;
            if (vec_out && e0 >= 0 && e0 + N <= V)
                *reinterpret_cast<uint4 *>(dx + e0) = E::pack(f);
            else
                store_edge(dx, e0, V, E::pack(f));
        };
        const int64_t tgt = target;
        const bool live = live_row(target, weight);
        // what the next iteration and the copies ahead need, loaded early
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
        if (!live) {
            if (rank == 0 && t == 0) {
                p.lp[row] = 0.0f;
                if (p.lse)
                    p.lse[row] = 0.0f;
                if (p.loss)
                    p.loss[row] = 0.0f;
            }
            if (dx) {
                float2 z[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j)
                    z[j] = make_float2(0.0f, 0.0f);
                for (int u = u0 + t; u < u1; u += blockDim.x)
                    store(u, z);
            }
        }
        const int par = nlive & 1;
        const uint32_t pph = (uint32_t)(nlive >> 1) & 1u;
        uint4 v[NV];
        float xt = 0.0f;
        RowInputs in = {};
        if (live) {
            if (warp == 0) {
                xt = E::load(x + tgt);  // before any CTA of the cluster writes the row (below)
                if (p.adv) {
                    in.old = p.lp_old[row];
                    in.adv = p.adv[row];
                    in.weight = p.weight[row];
                    in.behav = p.lp_behav ? p.lp_behav[row] : 0.0f;
                    in.ref = p.lp_ref ? p.lp_ref[row] : 0.0f;
                    in.hi = p.clip_hi ? p.clip_hi[row] : 1.0f + p.eps_hi;
                }
            }
            const int buf = nlive % bufs;
            // (a wait that runs out is reported by rlq_check; the loop goes on, without
            // waiting, so that the cluster's CTAs end together)
            if (!*abort_flag)
                mbar_wait(smem_u32(&bars[buf]), (uint32_t)(nlive / bufs) & 1u, abort_flag, plan.timeout_ns,
                          SITE_LOSS_ROW);
            const uint4 *src = reinterpret_cast<const uint4 *>(data) + buf * cap;
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = t + i * (int)blockDim.x;
                constexpr uint32_t ninf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
                v[i] = u0 + u < u1 ? src[u] : make_uint4(ninf, ninf, ninf, ninf);
                m = E::max_of(m, v[i]);
            }
            // a part that is all -inf sums zeros against any finite maximum
            const float mm = m == -INFINITY ? 0.0f : m;
            const float2 nm2 = make_float2(-mm, -mm);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 f = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), nm2), c2);
                    sum = __fadd2_rn(sum, make_float2(ex2(f.x), ex2(f.y)));
                }
            float S = sum.x + sum.y, wm = m;
#pragma unroll
            for (int o = 16; o; o >>= 1)
                wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, o));
            S = S == 0.0f ? 0.0f : S * ex2((m - wm) * c);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                S += __shfl_xor_sync(0xFFFFFFFFu, S, o);
            // A NaN target makes the sum NaN whichever warp holds it; this also has the
            // first warp's arrival, and so any write to the row, wait for the load of xt.
            if (warp == 0 && xt != xt)
                S = xt;
            if (lane == 0)
                pairs[par][warp] = make_float2(wm, S);
            __syncwarp();
            // The pairs of this parity are written again two rows on, behind the next
            // row's barrier, which the warps that read them reach afterwards.
            if (csize > 1)
                cluster_arrive();
            else
                __syncthreads();
        }
        const bool more = live_row(ahead_target, ahead_weight);
        if (live && csize > 1)
            cluster_wait();
        // Behind the barrier every warp has its part of the row in registers: the row's
        // buffer takes a later one.  (An empty row's: the last live row's is free since then.)
        if (more && t == 0)
            issue(ahead, ahead_live % bufs);
        if (warp == 0 && live) {
            float2 o[MAX_CLUSTER * MAX_WARPS / 32];
            float gm = -INFINITY, G = 0.0f;
#pragma unroll
            for (int k = 0; k < MAX_CLUSTER * MAX_WARPS / 32; ++k) {
                // entry e: warp e % 16 of rank e / 16 (the same order in every CTA)
                const int e = lane + 32 * k, r = e / MAX_WARPS, w = e % MAX_WARPS;
                o[k] = make_float2(-INFINITY, 0.0f);
                if (r < csize && w < nw)
                    o[k] = csize > 1 ? ld_cluster2(smem_u32(&pairs[par][w]), r) : pairs[par][w];
                gm = fmaxf(gm, o[k].x);
            }
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
            const RowScalars r = row_scalars(p, in, gm, G, xt, c);
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
        }
        if (live && dx) {
            if (!*abort_flag)
                mbar_wait(smem_u32(&coef_bars[par]), pph, abort_flag, plan.timeout_ns, SITE_LOSS_ROW);
            __syncwarp();
        }
        T raw[N];
        int eu = -1;
        if (more && warp == nw - 1) {
            const T *xa = logits + ahead * p.ld;
            eu = edge_unit(xa);
            if (eu >= 0)
                load_edge(xa, eu * N - offset(xa), V, raw);
        }
        if (live && dx) {
            const float4 k4 = coef[par];
            const float2 f2 = make_float2(k4.x, k4.x), ng2 = make_float2(-k4.y, -k4.y);
            const int te = (int)tgt + off, ut = te / N, jt = te - ut * N;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = u0 + t + i * (int)blockDim.x;
                if (u < u1) {
                    float2 f[N / 2];
#pragma unroll
                    for (int j = 0; j < N / 2; ++j) {
                        const float2 z = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), ng2), c2);
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
                    store(u, f);
                }
            }
        }
        if (more) {
            if (warp == nw - 1) {
                if (eu >= 0) {
                    reinterpret_cast<uint4 *>(data)[(ahead_live % bufs) * cap + eu - u0] = join_edge<T>(raw);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&bars[ahead_live % bufs]));
            }
            ++ahead_live;
        }
        if (live)
            ++nlive;
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

template <typename T, int NV, int kThreads>
cudaError_t launch_rows(const PolicyLossArgs &p, RowsPlan plan, int threads, cudaStream_t st)
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
    auto kernel = k_policy_rows<T, NV, kThreads>;
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
cudaError_t launch_typed(const PolicyLossArgs &p, cudaStream_t st)
{
    constexpr int N = Elem<T>::N;
    const int64_t units = (p.V + N - 1) / N + 1;  // one more where the rows start off a boundary
    // a row in one CTA of at most 256 threads x 8 units (32 KB), else in the smallest
    // cluster whose CTAs hold that, else in a cluster of 8 with more per CTA
    int csize = 1;
    while (csize < MAX_CLUSTER && units > (int64_t)csize * 256 * 8)
        csize *= 2;
    RowsPlan plan;
    plan.csize = csize;
    plan.units_cta = (int)((units + csize - 1) / csize);
    plan.timeout_ns = wait_limit_ns();
    const int64_t row = (int64_t)plan.units_cta * 16;
    // two CTAs per SM where that leaves each two rows at least, else one
    const int64_t room = 4 * row <= SMEM_CTA ? SMEM_CTA / 2 : SMEM_CTA;
    plan.bufs = (int)(room / row < MAX_BUFS ? room / row : MAX_BUFS);
    const int threads = plan.units_cta >= 256 * 16 ? 512 : plan.units_cta >= 256 ? 256 : (plan.units_cta + 31) / 32 * 32;
    const int nv = (plan.units_cta + threads - 1) / threads;
    if (threads == 512)
        return launch_rows<T, 16, 512>(p, plan, threads, st);
    return nv <= 1   ? launch_rows<T, 1, 256>(p, plan, threads, st)
           : nv <= 2 ? launch_rows<T, 2, 256>(p, plan, threads, st)
           : nv <= 4 ? launch_rows<T, 4, 256>(p, plan, threads, st)
           : nv <= 8 ? launch_rows<T, 8, 256>(p, plan, threads, st)
                     : launch_rows<T, 16, 256>(p, plan, threads, st);
}

}  // namespace

int64_t policy_max_vocab(int dtype) { return (int64_t)8 * 512 * 16 * (dtype == RLQ_DTYPE_F32 ? 4 : 8) - 8; }

cudaError_t take_loss_error_word(cudaStream_t st, unsigned long long *word) { return take_error_word(st, word); }

cudaError_t launch_policy_rows(const PolicyLossArgs &p, cudaStream_t st)
{
    return p.dtype == RLQ_DTYPE_F32 ? launch_typed<uint32_t>(p, st) : launch_typed<uint16_t>(p, st);
}

}  // namespace rlq
