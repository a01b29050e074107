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
// Bound by memory: the logits are read once and the gradient written once.  A CTA streams
// its row (few rows: a cluster its row, a part each) once for the maximum and the sum,
// and once more, from L2, for the gradient.  The rows in flight, two a SM at most, are
// 78 MB at 128256 bf16 logits, within the 129 MB of L2; the second pass runs backwards,
// from what was read last, and stores the gradient as streaming data.  The gradient may
// overwrite the logits: a thread reads what it overwrites, and a cluster's CTAs read the
// target's logit before any of them writes.
//
// Measured with the gradient, 15% of the rows empty and so not read: 4096 rows of 128256
// bf16 365 us (0.78 of the HBM rate) or 394 (0.72; which of the two goes with the block of
// memory that the gradient is written to), 2048 x 32000 fp32 83 us (0.86), 2048 x 151936
// bf16 227 us (0.75).  Without it, every row read: 2048 x 128256 bf16 83 us (0.93).
// Holding rows on chip instead (clusters of up to 8 CTAs, rows copied ahead to shared
// memory, a joining and a copying warp beside the reducing ones), which reads the logits
// from L2 once, took 439, 97 and 367 us: a row's chain of barriers and remote reads, with
// few warps a SM, cost more than the second read.
#include <cuda_runtime.h>

#include "rlq_internal.h"
#include "rlq_rows.cuh"

namespace rlq {
namespace {

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
    const float lr = o.lp - in.old, rho = expf(lr);
    // (minima by comparison: a NaN among the row's inputs stays one, fminf would drop it)
    float isw = 1.0f;
    if (p.lp_behav) {
        const float w = expf(in.old - in.behav);
        isw = w > p.tis_cap ? p.tis_cap : w;
    }
    float clip = rho < 1.0f - p.eps_lo ? 1.0f - p.eps_lo : rho;
    clip = clip > in.hi || in.hi != in.hi ? in.hi : clip;
    // (no advantage: 0, also where a finite ratio's exponential overflows)
    const float plain = in.adv == 0.0f && lr < INFINITY ? 0.0f : rho * in.adv, clipped = clip * in.adv;
    float loss = -isw * (plain > clipped || clipped != clipped ? clipped : plain);
    float dlp = plain > clipped ? 0.0f : -isw * plain;
    if (p.lp_ref) {
        const float d = in.ref - o.lp, e = expm1f(d);
        if (p.kl_beta > 0.0f || d != d) {  // (0 switches the term off, even where e overflows)
            loss = fmaf(p.kl_beta, e - d, loss);
            dlp = fmaf(-p.kl_beta, e, dlp);
        }
    }
    o.loss = in.weight * loss;
    o.dlp = in.weight * dlp;
    return o;
}

constexpr int MAX_CLUSTER = 8;

// Threads of a full CTA, and CTAs per SM.  Without the gradient more, smaller CTAs: 600
// rows of 32001 fp32 logits 14.6 us, with 512 threads 15.6 (2048 of 128256 bf16: 82.9 and
// 81.5).
template <bool kGrad>
constexpr int THREADS = kGrad ? 512 : 256;
template <bool kGrad>
constexpr int CTAS_SM = kGrad ? 2 : 4;

// Units are a row's 16-byte pieces on 16-byte boundaries: unit u covers elements u N - off
// .. + N - 1, off being the elements by which the row starts past a boundary.  The CTA of
// rank c of a row's cluster takes units c units_cta .. (c + 1) units_cta - 1, its threads
// in turn, BATCH loads of 16 bytes a thread in flight.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(THREADS<kGrad>, CTAS_SM<kGrad>)
    k_token_rows(const PolicyLossArgs p, int csize, int units_cta)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N, BATCH = 8, BATCH_GRAD = 4;
    constexpr uint32_t NINF = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    __shared__ float2 pairs[THREADS<kGrad> / 32], mine;
    __shared__ float4 coef;  // -dz / sum, the maximum, dz
    const int64_t row = blockIdx.x / csize;
    const int rank = (int)(blockIdx.x - row * csize), V = (int)p.V;
    const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5, nw = threads >> 5;
    const T *x = reinterpret_cast<const T *>(p.logits) + row * p.ld;
    T *dx = kGrad ? reinterpret_cast<T *>(p.dlogits) + row * p.ldd : nullptr;
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int u0 = rank * units_cta, u1 = min(u0 + units_cta, (off + V + N - 1) / N);
    const int whole0 = off ? 1 : 0, whole1 = (off + V) / N;  // units that the row's ends do not cut
    // the gradient's rows share the logits' 16-byte phase: whole units leave as one store
    const bool vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    auto store = [&](int u, uint4 v) {
        if (vec && u >= whole0 && u < whole1)
            __stcs(reinterpret_cast<uint4 *>(dx + ((int64_t)u * N - off)), v);
        else
            store_cut(dx, u * N - off, V, v);
    };
    auto load = [&](int u) {
        if (u >= u1)
            return make_uint4(NINF, NINF, NINF, NINF);
        return u >= whole0 && u < whole1 ? ld_row(x + ((int64_t)u * N - off)) : load_cut(x, u * N - off, V);
    };

    const int64_t target = p.targets[row];
    if (target < 0 || target >= V || (p.weight && p.weight[row] == 0.0f)) {  // an empty row, to the whole cluster
        if (rank == 0 && t == 0) {
            p.lp[row] = 0.0f;
            if (p.lse)
                p.lse[row] = 0.0f;
            if (p.loss)
                p.loss[row] = 0.0f;
        }
        if (kGrad)
            for (int u = u0 + t; u < u1; u += threads)
                store(u, make_uint4(0, 0, 0, 0));
        return;
    }
    const bool joins = warp == 0 && (kGrad || rank == 0);  // with the gradient every CTA needs the row's factors
    float xt = 0.0f;
    RowInputs in = {};
    if (joins) {
        xt = E::load(x + target);
        in = row_inputs(p, row);
    }
    const float c = 1.4426950408889634f / p.temperature;
    const float2 c2 = make_float2(c, c);
    float m = -INFINITY;
    float2 sum = make_float2(0.0f, 0.0f);
    for (int u = u0 + t; u < u1; u += BATCH * threads) {
        uint4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            v[i] = load(u + i * threads);
        float b = m;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            b = E::max_of(b, v[i]);
        if (b > m) {  // (m = -inf: the sum is 0, or NaN, so far)
            const float k = m == -INFINITY ? 1.0f : ex2((m - b) * c);
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
                sum = __fadd2_rn(sum, make_float2(ex2(f.x), ex2(f.y)));
            }
    }
    float2 o = join_pairs(make_float2(m, sum.x + sum.y), c);
    // A NaN target makes the sum NaN whichever thread holds it; this also has this warp's
    // pair, and so any write to the row, wait for the load of xt.
    if (joins && xt != xt)
        o.y = xt;
    if (lane == 0)
        pairs[warp] = o;
    __syncthreads();
    if (warp == 0) {
        o = join_pairs(lane < nw ? pairs[lane] : make_float2(-INFINITY, 0.0f), c);
        if (lane == 0)
            mine = o;
        __syncwarp();
    }
    if (csize > 1) {
        cluster_arrive();
        cluster_wait();
        if (joins)
            o = join_pairs(lane < csize ? ld_cluster2(&mine, lane) : make_float2(-INFINITY, 0.0f), c);
        __syncwarp();
    }
    if (joins) {
        const RowScalars r = row_scalars(p, in, o.x, o.y, xt, c);
        if (lane == 0) {
            if (kGrad) {
                // -dz * softmax; an empty row's probabilities are 0
                const float dz = r.dlp / p.temperature;
                coef = make_float4(o.y == 0.0f ? 0.0f : -dz / o.y, o.x == -INFINITY ? 0.0f : o.x, dz, 0.0f);
            }
            if (rank == 0) {
                p.lp[row] = r.lp;
                if (p.lse)
                    p.lse[row] = r.lse;
                if (p.loss)
                    p.loss[row] = r.loss;
            }
        }
        __syncwarp();
    }
    if (csize > 1)
        cluster_arrive_relaxed();  // this CTA has read the others' pairs
    if (kGrad) {
        __syncthreads();
        const float4 k4 = coef;
        const float2 f2 = make_float2(k4.x, k4.x), ng2 = make_float2(-k4.y, -k4.y);
        const int te = (int)target + off, ut = te / N, jt = te - ut * N;
        const int step = BATCH_GRAD * threads;
        for (int u = u0 + t + (u1 - u0 - 1) / step * step; u >= u0; u -= step) {
            uint4 v[BATCH_GRAD];
#pragma unroll
            for (int i = 0; i < BATCH_GRAD; ++i)
                v[i] = load(u + i * threads);
#pragma unroll
            for (int i = 0; i < BATCH_GRAD; ++i) {
                const int w = u + i * threads;
                if (w >= u1)
                    break;
                float2 f[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 z = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), ng2), c2);
                    f[j] = __fmul2_rn(make_float2(ex2(z.x), ex2(z.y)), f2);
                }
                if (w == ut) {
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j == jt) {
                            if (j & 1)
                                f[j / 2].y += k4.z;
                            else
                                f[j / 2].x += k4.z;
                        }
                }
                store(w, E::pack(f));
            }
        }
    }
    if (csize > 1)
        cluster_wait();  // no CTA leaves while another may still read its pair
}

template <typename T, bool kGrad>
cudaError_t launch_rows(const PolicyLossArgs &p, cudaStream_t st)
{
    constexpr int N = Elem<T>::N;
    const int64_t units = (p.V + N - 1) / N + 1;  // one more where the rows start off a boundary
    // A row to a cluster where there are too few to fill the SMs and a thread keeps two
    // units, while the clusters of all rows are resident with room to spare (512 and more
    // of them compete for the SMs that have a whole cluster's room: 600 rows of 32001 fp32
    // logits 14.6 us in single CTAs, 18.0 in pairs; 152 rows 5.7 in pairs, 7.3 in fours).
    const int64_t slots = (int64_t)CTAS_SM<kGrad> * device_sms();
    int csize = 1;
    while (csize < MAX_CLUSTER && (kGrad ? 2 : 3) * p.rows * csize <= slots &&
           units >= (int64_t)csize * 4 * THREADS<kGrad>)
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
    cfg.blockDim = dim3(units_cta >= THREADS<kGrad> ? THREADS<kGrad> : (units_cta + 31) / 32 * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_token_rows<T, kGrad>, p, csize, units_cta);
}

}  // namespace

cudaError_t launch_policy_rows(const PolicyLossArgs &p, cudaStream_t st)
{
    if (p.dtype == RLQ_DTYPE_F32)
        return p.dlogits ? launch_rows<uint32_t, true>(p, st) : launch_rows<uint32_t, false>(p, st);
    return p.dlogits ? launch_rows<uint16_t, true>(p, st) : launch_rows<uint16_t, false>(p, st);
}

}  // namespace rlq
