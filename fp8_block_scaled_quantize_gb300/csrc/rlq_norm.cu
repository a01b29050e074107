// Residual addition + RMSNorm + FP8 quantizer, and the norm's backward pass (sm_103a).
//
// Forward, per row m of the residual stream:
//   h = bf16_RN(res + delta)                     written back, the stream is held in bf16
//   rstd = 1 / sqrt(mean(h^2) + eps)             fp32, the sum taken over h as stored
//   x = (h * rstd) * gamma                       fp32, not rounded before it is quantized
//   1x128 codes and scales of x (and 128x1, transposed, for WGrad)
// Backward, with xh = h * rstd and dn = dx * gamma:
//   dh = dres + rstd * (dn - xh * mean(dn * xh)),   dgamma = sum_m dx * xh
//
// Both are bound by memory: 7.03 bytes per element forward (2 + 2 read, 2 + 1 and a
// scale per 128 written; 8.06 with the 128x1 codes), 8 backward.  Measured at 8192 x 4096:
// forward 38.6 us (0.90 of the HBM rate; 0.95 at 16384 x 5120; 40 us with unpacked fp32 arithmetic, whose
// instructions filled 0.72 of the issue slots); with the 128x1 codes 54.7 us, since the
// column groups need every row's factor first and read h again (2 bytes an element: 10
// us, of which L2 saves little); backward 47.5 us (0.83).  Tried for the second read and slower or
// equal: row blocks in the order that was written last, both passes over chunks of rows
// that fit L2 (64-88 us), L2 hints on the inputs (62 us).
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"

namespace rlq {
namespace {

constexpr int GRP = 128;
constexpr int MAX_K = 16384;  // (the entry points refuse more)

// A load that may alias an output of the same kernel (read by the thread that
// later overwrites it), so not through the read-only path.
__device__ __forceinline__ uint4 ld_once(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Sums of two bf16 pairs, rounded once.  (The same bits as an fp32 sum rounded to bf16:
// that sum is exact unless the exponents are more than 16 apart, and then both are the
// larger term.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 8 bf16 as four pairs of fp32.
__device__ __forceinline__ void unpack4x2(const uint4 &v, float2 (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(bf_lo(w[i]), bf_hi(w[i]));
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Sum over the threads of one team: warps `w0 ..` of `nw` warps, partials in `sh`
// (nw floats), named barrier `bar` of 32 * nw threads.  Every thread gets the sum,
// added in the same order in each.  `sh` may be reused after the next barrier.
__device__ __forceinline__ float team_sum(float v, float *sh, int wi, int nw, int bar)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (nw == 1)
        return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
        sh[wi] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * nw) : "memory");
    v = lane < nw ? sh[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One CTA per row; thread t holds the 16-byte vectors t + i * blockDim.x, i < NV,
// all loads in flight before the sum.  A 1x128 group is 16 consecutive lanes of one
// vector index.
template <int NV, bool kAdd>
__global__ void __launch_bounds__(1024) k_add_rmsnorm_rows(const uint16_t *res, int64_t ldr, const uint16_t *delta, int64_t ldd,
                                   const uint16_t *__restrict__ gamma, float eps, int K, uint16_t *h, int64_t ldh,
                                   float *__restrict__ rstd, uint8_t *__restrict__ q, int64_t ldq,
                                   float *__restrict__ s, int64_t lds)
{
    pdl_begin();
    __shared__ float sh[32];
    const int64_t m = blockIdx.x;
    const int t = threadIdx.x, T = blockDim.x, nvec = K / 8;
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * T;
        v[i] = c < nvec ? ld_once(res + m * ldr + 8 * c) : make_uint4(0, 0, 0, 0);
    }
    if (kAdd) {
        uint4 d[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * T;
            d[i] = c < nvec ? ld_once(delta + m * ldd + 8 * c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = make_uint4(add_bf16x2(v[i].x, d[i].x), add_bf16x2(v[i].y, d[i].y), add_bf16x2(v[i].z, d[i].z),
                              add_bf16x2(v[i].w, d[i].w));
    }
    float2 ss2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * T;
        if (h && c < nvec)
            *reinterpret_cast<uint4 *>(h + m * ldh + 8 * c) = v[i];
        float2 f[4];
        unpack4x2(v[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ss2 = __ffma2_rn(f[j], f[j], ss2);
    }
    const float ss = team_sum(ss2.x + ss2.y, sh, t >> 5, T >> 5, 0);
    const float r = __frcp_rn(__fsqrt_rn(ss / (float)K + eps));
    if (t == 0)
        rstd[m] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * T;
        const bool in = c < nvec;
        float2 f[4], g[4];
        unpack4x2(v[i], f);
        unpack4x2(in ? *reinterpret_cast<const uint4 *>(gamma + 8 * c) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[j] = __fmul2_rn(__fmul2_rn(f[j], both(r)), g[j]);
        const float sc = group_scale(half_warp_max(max_abs8(f)));
        if (in) {
            if ((t & 15) == 0)
                s[(int64_t)(c >> 4) * lds + m] = sc;
            *reinterpret_cast<uint2 *>(q + m * ldq + 8 * c) = encode8f(f, scale_pre(sc), scale_rcp(sc));
        }
    }
}

// The 128x1 groups of the same x, read back from h and rstd: a CTA takes a 128 x 128
// tile, thread t rows 8 (t / 16) .. + 7 and columns 8 (t % 16) .. + 7.  The codes
// are turned in shared memory ([column][16 chunks of 8 rows], chunks XOR-swizzled by
// column / 8: conflict-free both ways) and leave as whole 128-byte lines of qT.
__global__ void __launch_bounds__(256, 3) k_norm_cols(const uint16_t *__restrict__ h, int64_t ldh,
                                                   const float *__restrict__ rstd,
                                                   const uint16_t *__restrict__ gamma, int64_t M, int64_t K,
                                                   uint8_t *__restrict__ qT, int64_t ldqT, float *__restrict__ sc,
                                                   int64_t ldsc)
{
    pdl_begin();
    __shared__ __align__(16) uint8_t tile[128 * 128];
    __shared__ __align__(16) float part[8][128];
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4, warp = t >> 5;
    const int64_t m0 = (int64_t)blockIdx.x * GRP, k0 = (int64_t)blockIdx.y * GRP;
    const int rows = (int)(M - m0 < GRP ? M - m0 : GRP);
    uint4 v[8];
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = 8 * rg + i;
        v[i] = m < rows ? ld_stream(h + (m0 + m) * ldh + k0 + 8 * cg) : make_uint4(0, 0, 0, 0);
        r[i] = m < rows ? rstd[m0 + m] : 0.0f;
    }
    const uint4 gv = *reinterpret_cast<const uint4 *>(gamma + k0 + 8 * cg);
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
    float2 x[8][4];  // [row][column pair]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[i][j] = __fmul2_rn(__fmul2_rn(make_float2(bf_lo(w[j]), bf_hi(w[j])), make_float2(r[i], r[i])),
                                 make_float2(bf_lo(gw[j]), bf_hi(gw[j])));
    }
    float2 cmax[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        cmax[j] = make_float2(max3_abs(x[0][j].x, x[1][j].x, x[2][j].x), max3_abs(x[0][j].y, x[1][j].y, x[2][j].y));
        cmax[j] = make_float2(max3_abs(cmax[j].x, x[3][j].x, x[4][j].x), max3_abs(cmax[j].y, x[3][j].y, x[4][j].y));
        cmax[j] = make_float2(max3_abs(cmax[j].x, x[5][j].x, x[6][j].x), max3_abs(cmax[j].y, x[5][j].y, x[6][j].y));
        cmax[j] = make_float2(fmaxf(cmax[j].x, fabsf(x[7][j].x)), fmaxf(cmax[j].y, fabsf(x[7][j].y)));
    }
    store_column_maxima(cmax, t & 16, part[warp] + 8 * cg);
    __syncthreads();
    float cs = 1.0f;
    if (t < 128) {
        float a = part[0][t];
#pragma unroll
        for (int w = 1; w < 8; ++w)
            a = fmaxf(a, part[w][t]);
        cs = group_scale(a);
        part[0][t] = scale_rcp(cs);  // (only this thread reads column t of the maxima)
        sc[(int64_t)blockIdx.x * ldsc + k0 + t] = cs;
    }
    // (columns whose scale is below 2^-100 are scaled up first)
    if (__syncthreads_or(cs < 0x1p-100f)) {
        if (t < 128)
            part[1][t] = scale_pre(cs);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = *reinterpret_cast<const float2 *>(part[1] + 8 * cg + 2 * j);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i][j] = __fmul2_rn(x[i][j], f);
        }
    }
    const float4 r0 = *reinterpret_cast<const float4 *>(part[0] + 8 * cg);
    const float4 r1 = *reinterpret_cast<const float4 *>(part[0] + 8 * cg + 4);
    const float2 rc[4] = {make_float2(r0.x, r0.y), make_float2(r0.z, r0.w), make_float2(r1.x, r1.y),
                          make_float2(r1.z, r1.w)};
    uint8_t *out = tile + 8 * cg * GRP + 8 * (rg ^ cg);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = __fmul2_rn(x[i][j], rc[j]);
        *reinterpret_cast<uint2 *>(out + 2 * j * GRP) =
            make_uint2(e4m3x4(y[0].x, y[1].x, y[2].x, y[3].x),
                       e4m3x4(y[4].x, y[5].x, y[6].x, y[7].x));
        *reinterpret_cast<uint2 *>(out + (2 * j + 1) * GRP) =
            make_uint2(e4m3x4(y[0].y, y[1].y, y[2].y, y[3].y),
                       e4m3x4(y[4].y, y[5].y, y[6].y, y[7].y));
    }
    __syncthreads();
    store_tile_T(tile, t, 256, rows, qT + k0 * ldqT + m0, ldqT);
}

// Backward.  A CTA holds `teams` teams of T threads; a team takes rows
// blockIdx.x * teams + team, + gridDim.x * teams, ..., each thread the same columns of
// every row, so the norm weight's gradient adds up in registers.  The next row's loads
// are in flight while this row is reduced and written (NV == 2; four vectors a thread
// leave no registers for it).  The teams' sums are added in
// team order in shared memory and leave as one partial row per CTA (or as dgamma
// itself from a single CTA); k_dgamma_sum adds the partial rows in order.
template <int NV>
__global__ void __launch_bounds__(512)
    k_rmsnorm_bwd(const uint16_t *__restrict__ dx, int64_t lddx, const uint16_t *__restrict__ h, int64_t ldh,
                  const float *__restrict__ rstd, const uint16_t *__restrict__ gamma, const uint16_t *dres,
                  int64_t lddres, uint16_t *dh, int64_t lddh, float *__restrict__ dgamma_part, int M, int K, int T,
                  int teams)
{
    pdl_begin();
    extern __shared__ float dyn[];  // K sums
    __shared__ float sh[2][32];
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int nvec = K / 8, nw = T >> 5, wi = t >> 5;
    const int step = gridDim.x * teams;
    float2 acc[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = both(0.0f);
    uint4 a[NV], b[NV], d[NV];
    float r = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load = [&](int m) {
        const bool row = m < M;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * T;
            const bool in = row && c < nvec;
            a[i] = in ? ld_stream(dx + (int64_t)m * lddx + 8 * c) : zero;
            b[i] = in ? ld_stream(h + (int64_t)m * ldh + 8 * c) : zero;
            d[i] = in && dres ? ld_once(dres + (int64_t)m * lddres + 8 * c) : zero;
        }
        r = row ? rstd[m] : 0.0f;
    };
    int m = blockIdx.x * teams + team;
    if (NV == 2)
        load(m);
    for (int par = 0; m < M; m += step, par ^= 1) {
        if (NV != 2)
            load(m);
        uint4 ca[NV], cb[NV], cd[NV];
        const float cr = r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ca[i] = a[i];
            cb[i] = b[i];
            cd[i] = d[i];
        }
        if (NV == 2)
            load(m + step < M ? m + step : M);
        float2 dot2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * T;
            float2 x[4], y[4], g[4];
            unpack4x2(ca[i], x);
            unpack4x2(cb[i], y);
            unpack4x2(c < nvec ? __ldg(reinterpret_cast<const uint4 *>(gamma + 8 * c)) : zero, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 xh = __fmul2_rn(y[j], both(cr));
                acc[i][j] = __ffma2_rn(x[j], xh, acc[i][j]);
                dot2 = __ffma2_rn(__fmul2_rn(x[j], g[j]), xh, dot2);
            }
        }
        // (the parity keeps a fast warp's next partials apart from the ones being read)
        const float dot = team_sum(dot2.x + dot2.y, sh[par] + team * nw, wi, nw, 1 + team) / (float)K;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * T;
            if (c >= nvec)
                continue;
            float2 x[4], y[4], g[4], e[4];
            unpack4x2(ca[i], x);
            unpack4x2(cb[i], y);
            unpack4x2(__ldg(reinterpret_cast<const uint4 *>(gamma + 8 * c)), g);
            unpack4x2(cd[i], e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 xh = __fmul2_rn(y[j], both(cr));
                e[j] = __ffma2_rn(both(cr), __ffma2_rn(xh, both(-dot), __fmul2_rn(x[j], g[j])), e[j]);
            }
            *reinterpret_cast<uint4 *>(dh + (int64_t)m * lddh + 8 * c) =
                make_uint4(pack_bf16x2(e[0]), pack_bf16x2(e[1]), pack_bf16x2(e[2]), pack_bf16x2(e[3]));
        }
    }
    for (int k = 0; k < teams; ++k) {
        if (team == k) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = t + i * T;
                if (c >= nvec)
                    continue;
                float4 *p = reinterpret_cast<float4 *>(dyn + 8 * c);
                float4 lo = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
                float4 hi = make_float4(acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y);
                if (k > 0) {
                    const float4 x = p[0], y = p[1];
                    lo = make_float4(lo.x + x.x, lo.y + x.y, lo.z + x.z, lo.w + x.w);
                    hi = make_float4(hi.x + y.x, hi.y + y.y, hi.z + y.z, hi.w + y.w);
                }
                p[0] = lo;
                p[1] = hi;
            }
        }
        __syncthreads();
    }
    float *out = dgamma_part + (int64_t)blockIdx.x * K;
    for (int c = threadIdx.x; c < K; c += blockDim.x)
        out[c] = dyn[c];
}

// dgamma[c] = sum over p < parts, in a fixed order, of part[p][c]: a CTA takes 32
// columns, warp w the partial rows w, w + 32, ..., all its loads in flight (one partial
// row a SM: five), and the warps' sums are added as a tree.  With eight warps, each
// 19 loads a few at a time, the pass took 1.6 us more (8192 x 4096: 48.8 -> 47.2 in all).
__global__ void __launch_bounds__(1024) k_dgamma_sum(const float *__restrict__ part, int parts, int K,
                                                     float *__restrict__ dgamma)
{
    pdl_begin();
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // K % 128 == 0: always in range
    float v = 0.0f;
    for (int p0 = w; p0 < parts; p0 += 8 * 32) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a[i] = p0 + 32 * i < parts ? part[(int64_t)(p0 + 32 * i) * K + c] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += a[i];
    }
    sh[w][lane] = v;
    __syncthreads();
    v = sh[lane][w];  // column w of this CTA, partial sum `lane`
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0)
        dgamma[blockIdx.x * 32 + w] = v;
}

// Launch shape of the backward kernel.
struct BwdPlan {
    int nv, T, teams, grid;
};

BwdPlan bwd_plan(int64_t M, int64_t K)
{
    BwdPlan p;
    const int nvec = (int)(K / 8);
    p.nv = K <= 8192 ? 2 : 4;
    p.T = ((nvec + p.nv - 1) / p.nv + 31) / 32 * 32;
    p.teams = p.T >= 512 ? 1 : (512 / p.T > 8 ? 8 : 512 / p.T);  // named barriers 1..8
    if (p.teams > M)
        p.teams = (int)M;
    const int64_t want = (M + p.teams - 1) / p.teams;
    const int sms = device_sms();
    p.grid = (int)(want < sms ? want : sms);
    return p;
}

}  // namespace

cudaError_t launch_add_rmsnorm_quant(const uint16_t *res, int64_t ldr, const uint16_t *delta, int64_t ldd, int64_t M,
                                     int64_t K, const uint16_t *gamma, float eps, uint16_t *h, int64_t ldh, float *rstd,
                                     uint8_t *q, int64_t ldq, float *s, int64_t lds, uint8_t *qT, int64_t ldqT,
                                     float *sc, int64_t ldsc, cudaStream_t st)
{
    // Vectors per thread.  As many rows as SMs or fewer: one, the shortest path through a
    // row.  More: two up to K = 5120 (M = 1001, K = 5120 7.3 us, with four 8.8), four
    // beyond, where a row's sum over more warps costs more (M = 4096, K = 8192 with the
    // columns 62 us, with two 68).
    const int nvec = (int)(K / 8);
    const int nv = (M <= device_sms() && nvec <= 1024) ? 1 : nvec <= 640 ? 2 : 4;
    const int T = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    auto kernel = nv == 1   ? (delta ? k_add_rmsnorm_rows<1, true> : k_add_rmsnorm_rows<1, false>)
                  : nv == 2 ? (delta ? k_add_rmsnorm_rows<2, true> : k_add_rmsnorm_rows<2, false>)
                            : (delta ? k_add_rmsnorm_rows<4, true> : k_add_rmsnorm_rows<4, false>);
    cudaError_t e = launch_pdl(kernel, dim3((unsigned)M), dim3(T), 0, st, res, ldr, delta, ldd, gamma, eps, (int)K, h,
                               ldh, rstd, q, ldq, s, lds);
    if (e != cudaSuccess || !qT)
        return e;
    const uint16_t *x = h ? h : res;
    return launch_pdl(k_norm_cols, dim3((unsigned)((M + GRP - 1) / GRP), (unsigned)(K / GRP)), dim3(256), 0, st, x,
                      h ? ldh : ldr, rstd, gamma, M, K, qT, ldqT, sc, ldsc);
}

int64_t rmsnorm_backward_ws_bytes(int64_t M, int64_t K)
{
    const BwdPlan p = bwd_plan(M, K);
    return p.grid > 1 ? (int64_t)p.grid * K * 4 : 0;
}

cudaError_t launch_rmsnorm_backward(const uint16_t *dx, int64_t lddx, const uint16_t *h, int64_t ldh, const float *rstd,
                                    const uint16_t *gamma, const uint16_t *dres, int64_t lddres, uint16_t *dh,
                                    int64_t lddh, float *dgamma, int64_t M, int64_t K, float *ws, cudaStream_t st)
{
    const BwdPlan p = bwd_plan(M, K);
    auto kernel = p.nv == 2 ? k_rmsnorm_bwd<2> : k_rmsnorm_bwd<4>;
    const size_t smem = (size_t)K * 4;
    // Four vectors a thread (K > 8192) may need more than the 48 KB, static and dynamic,
    // that a kernel has unasked.  The limit is the process's: raised once per device, to
    // the largest K's, and never lowered under another thread's launch.
    static std::atomic<bool> raised[64];
    int dev = 0;
    cudaError_t e = p.nv == 2 ? cudaSuccess : cudaGetDevice(&dev);
    if (e == cudaSuccess && p.nv != 2 && !raised[dev & 63].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_K * 4);
        raised[dev & 63].store(e == cudaSuccess, std::memory_order_relaxed);
    }
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(kernel, dim3(p.grid), dim3(p.T * p.teams), smem, st, dx, lddx, h, ldh, rstd, gamma, dres, lddres, dh,
                   lddh, p.grid > 1 ? ws : dgamma, (int)M, (int)K, p.T, p.teams);
    if (e != cudaSuccess || p.grid == 1)
        return e;
    return launch_pdl(k_dgamma_sum, dim3((unsigned)(K / 32)), dim3(1024), 0, st, ws, p.grid, (int)K, dgamma);
}

}  // namespace rlq
