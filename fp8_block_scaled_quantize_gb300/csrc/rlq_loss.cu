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
// held in the registers of one CTA, or of a cluster of 2, 4 or 8 for long rows, between
// the pass that takes the maximum, the one that sums the exponentials and the one that
// writes the gradient; the CTAs of a cluster exchange one (maximum, sum) pair each
// through distributed shared memory.  The gradient may overwrite the logits.
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"

namespace rlq {
namespace {

constexpr int MAX_THREADS = 512;

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

// 16 bytes that the same thread may overwrite later in the kernel.
__device__ __forceinline__ uint4 ld16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ float2 ld_cluster2(uint32_t a, uint32_t rank)
{
    uint32_t r;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(r) : "memory");
    return v;
}

struct RowScalars {
    float lp, lse, loss, dlp;
};

// The row's loss and its derivative, from the row's maximum (m, in logits), the sum S
// of 2^((x - m) c) and the target's logit.
__device__ __noinline__ RowScalars row_scalars(const PolicyLossArgs &p, int64_t row, float m, float S, float xt,
                                                  float c)
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
    const float old = p.lp_old[row], adv = p.adv[row], w = p.weight[row];
    const float rho = expf(o.lp - old);
    const float isw = p.lp_behav ? fminf(expf(old - p.lp_behav[row]), p.tis_cap) : 1.0f;
    const float hi = p.clip_hi ? p.clip_hi[row] : 1.0f + p.eps_hi;
    const float plain = rho * adv, clipped = fminf(fmaxf(rho, 1.0f - p.eps_lo), hi) * adv;
    float loss = -isw * fminf(plain, clipped);
    float dlp = plain <= clipped ? -isw * plain : 0.0f;
    if (p.lp_ref) {
        const float d = p.lp_ref[row] - o.lp, e = expm1f(d);
        loss = fmaf(p.kl_beta, e - d, loss);
        dlp = fmaf(-p.kl_beta, e, dlp);
    }
    o.loss = w * loss;
    o.dlp = w * dlp;
    return o;
}

// The unit at elements e0 .. of a row of V: elements outside the row read as -inf, and
// are not written.  (Out of line: a row has at most one such unit at each end.)
template <typename T>
__device__ __noinline__ uint4 load_edge(const T *x, int e0, int V)
{
    constexpr int N = Elem<T>::N;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (e0 + j >= 0 && e0 + j < V) {
            const uint32_t b = (uint32_t)x[e0 + j];
            if (sizeof(T) == 2)
                w[j / 2] = (j & 1) ? (w[j / 2] & 0xFFFFu) | (b << 16) : (w[j / 2] & 0xFFFF0000u) | b;
            else
                w[j & 3] = b;
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

// A cluster per row.  Units are the row's 16-byte pieces on 16-byte boundaries: unit u
// covers elements u N - off .. + N - 1, off being the elements by which the row starts
// past a boundary; elements outside the row read as -inf and are not written.  The CTA
// of rank c takes units c units_cta .. (c + 1) units_cta - 1, thread t of it units
// t + i * blockDim.x, i < NV.
template <typename T, int NV>
__global__ void __launch_bounds__(MAX_THREADS, NV <= 8 ? 2 : 1) k_policy_rows(const PolicyLossArgs p, int csize, int units_cta)
{
    pdl_begin();
    using E = Elem<T>;
    constexpr int N = E::N;
    __shared__ float red[2][16];
    __shared__ __align__(8) float2 mine;
    __shared__ float4 coef;
    const int64_t row = blockIdx.x / csize;
    const int rank = blockIdx.x - (int)(row * csize);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x >> 5;
    const T *x = reinterpret_cast<const T *>(p.logits) + row * p.ld;
    T *dx = p.dlogits ? reinterpret_cast<T *>(p.dlogits) + row * p.ldd : nullptr;
    const int V = (int)p.V;
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int u0 = rank * units_cta, u1 = min(u0 + units_cta, (off + V + N - 1) / N);
    // the gradient's rows share the logits' 16-byte phase: whole units leave as one store
    const bool vec_out = dx && ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    const int64_t target = p.targets[row];
    const bool skip = target < 0 || target >= V || (p.weight && p.weight[row] == 0.0f);

    auto store = [&](int u, const float2(&f)[N / 2]) {
        const int e0 = u * N - off;
        if (vec_out && e0 >= 0 && e0 + N <= V)
            *reinterpret_cast<uint4 *>(dx + e0) = E::pack(f);
        else
            store_edge(dx, e0, V, E::pack(f));
    };

    if (skip) {  // (the whole cluster: no exchange is left waiting)
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
        return;
    }

    const float xt = E::load(x + target);  // before any CTA of the cluster writes
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = u0 + t + i * (int)blockDim.x, e0 = u * N - off;
        if (u < u1 && e0 >= 0 && e0 + N <= V) {
            v[i] = ld16(x + e0);
        } else {
            v[i] = load_edge(x, u < u1 ? e0 : V, V);
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float2 f = E::get2(v[i], j);
            m = fmaxf(m, fmaxf(f.x, f.y));
        }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0)
        red[0][warp] = m;
    __syncthreads();
    m = lane < nw ? red[0][lane] : -INFINITY;
#pragma unroll
    for (int o = 8; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    m = __shfl_sync(0xFFFFFFFFu, m, 0);
    // a CTA whose part is all -inf sums zeros against any finite maximum
    const float mm = m == -INFINITY ? 0.0f : m;
    const float c = 1.4426950408889634f / p.temperature;
    const float2 c2 = make_float2(c, c), nm2 = make_float2(-mm, -mm);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float2 f = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), nm2), c2);
            sum = __fadd2_rn(sum, make_float2(ex2(f.x), ex2(f.y)));
        }
    float S = sum.x + sum.y;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        S += __shfl_xor_sync(0xFFFFFFFFu, S, o);
    if (lane == 0)
        red[1][warp] = S;
    __syncthreads();
    if (warp == 0) {
        S = lane < nw ? red[1][lane] : 0.0f;
#pragma unroll
        for (int o = 8; o; o >>= 1)
            S += __shfl_xor_sync(0xFFFFFFFFu, S, o);
        if (lane == 0)
            mine = make_float2(m, S);
    }
    if (csize > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
        __syncwarp();
        // (lane r holds rank r's pair; the sum goes in rank order in every CTA)
        float2 o = make_float2(-INFINITY, 0.0f);
        if (csize == 1) {
            if (lane == 0)
                o = mine;
        } else if (lane < csize) {
            o = ld_cluster2(smem_addr(&mine), lane);
        }
        float gm = o.x;
#pragma unroll
        for (int k = 4; k; k >>= 1)
            gm = fmaxf(gm, __shfl_xor_sync(0xFFFFFFFFu, gm, k));
        gm = __shfl_sync(0xFFFFFFFFu, gm, 0);
        // (a part of -inf only has the sum 0; one of NaN has no maximum but a NaN sum)
        const float part = o.y == 0.0f ? 0.0f : o.y * ex2((o.x - gm) * c);
        float G = 0.0f;
        for (int k = 0; k < csize; ++k)
            G += __shfl_sync(0xFFFFFFFFu, part, k);
        if (lane == 0) {
            const RowScalars r = row_scalars(p, row, gm, G, xt, c);
            const float dz = r.dlp / p.temperature;
            // gradient: -dz * softmax, softmax = 2^((x - mm) c) * 2^((mm - gm) c) / G
            // (a CTA whose part is all -inf has probabilities 0 only)
            coef = make_float4(S == 0.0f ? 0.0f : -dz * ex2((mm - gm) * c) / G, dz, 0.0f, 0.0f);
            if (rank == 0) {
                p.lp[row] = r.lp;
                if (p.lse)
                    p.lse[row] = r.lse;
                if (p.loss)
                    p.loss[row] = r.loss;
            }
        }
    }
    // the peers' pairs are read: a CTA leaves once all have said so (below)
    if (csize > 1) {
        __syncthreads();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (dx) {
        const float4 k = coef;
        const float2 f2 = make_float2(k.x, k.x);
        const int ut = (int)((target + off) / N), jt = (int)((target + off) - (int64_t)ut * N);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = u0 + t + i * (int)blockDim.x;
            if (u >= u1)
                break;
            float2 f[N / 2];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float2 z = __fmul2_rn(__fadd2_rn(E::get2(v[i], j), nm2), c2);
                f[j] = __fmul2_rn(make_float2(ex2(z.x), ex2(z.y)), f2);
            }
            if (u == ut) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j == jt) {
                        if (j & 1)
                            f[j / 2].y += k.y;
                        else
                            f[j / 2].x += k.y;
                    }
            }
            store(u, f);
        }
    }
    if (csize > 1)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int NV>
cudaError_t launch_rows(const PolicyLossArgs &p, int threads, int csize, int units_cta, cudaStream_t st)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.rows * csize));
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_policy_rows<T, NV>, p, csize, units_cta);
}

template <typename T>
cudaError_t launch_typed(const PolicyLossArgs &p, cudaStream_t st)
{
    constexpr int N = Elem<T>::N;
    const int64_t units = (p.V + N - 1) / N + 1;  // one more where the rows start off a boundary
    // a row in one CTA of at most 512 threads x 8 units (64 KB), else in the smallest
    // cluster whose CTAs hold that, else in a cluster of 8 with 16 units a thread
    int csize = 1;
    while (csize < 8 && units > (int64_t)csize * MAX_THREADS * 8)
        csize *= 2;
    const int per_cta = (int)((units + csize - 1) / csize);
    const int threads = per_cta >= MAX_THREADS ? MAX_THREADS : (per_cta + 31) / 32 * 32;
    const int nv = (per_cta + threads - 1) / threads;
    return nv <= 1   ? launch_rows<T, 1>(p, threads, csize, per_cta, st)
           : nv <= 2 ? launch_rows<T, 2>(p, threads, csize, per_cta, st)
           : nv <= 4 ? launch_rows<T, 4>(p, threads, csize, per_cta, st)
           : nv <= 8 ? launch_rows<T, 8>(p, threads, csize, per_cta, st)
                     : launch_rows<T, 16>(p, threads, csize, per_cta, st);
}

}  // namespace

int64_t policy_max_vocab(int dtype)
{
    return (int64_t)8 * MAX_THREADS * 16 * (dtype == RLQ_DTYPE_F32 ? 4 : 8) - 8;
}

cudaError_t launch_policy_rows(const PolicyLossArgs &p, cudaStream_t st)
{
    return p.dtype == RLQ_DTYPE_F32 ? launch_typed<uint32_t>(p, st) : launch_typed<uint16_t>(p, st);
}

}  // namespace rlq
