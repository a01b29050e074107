// Backward pass of the gated feed-forward block's activation, from the 8-bit
// checkpoint of its two projections (sm_103a).
//
// With g and u the checkpoint's values (code * scale), sg = 1 / (1 + exp(-g)):
//   dg = da * u * sg * (1 + g (1 - sg)),   du = da * g * sg,   a = g * sg * u
// and [dg | du] is one [M, 2F] gradient: its 1x128 codes feed DGrad, its 128x1 codes
// (transposed) WGrad, both over the stacked gate / up weight; the 128x1 codes of a are
// the down projection's WGrad operand, formed again here so that the forward pass
// keeps two bytes per column and no more.  Everything between the loads and the codes
// is fp32.
//
// Bound by memory: 2 + 1 + 1 bytes read and 2 + 2 + 1 written per element of [M, F].
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"

namespace rlq {
namespace {

constexpr int GRP = 128;
constexpr int THREADS = 512;
constexpr int TILE_BYTES = GRP * GRP;                            // one operand's transposed codes
constexpr int SMEM_BYTES = 3 * TILE_BYTES + 16 * 3 * GRP * 4;  // and 16 warps' column maxima

struct GateBwd {
    const uint16_t *da;
    int64_t ldda;
    const uint8_t *guq;
    int64_t ldguq;
    const float *gus;
    int64_t ld_gus;
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t lds;
    uint8_t *qT;
    int64_t ldqT;
    float *sc;
    int64_t ldsc;
    uint8_t *aT;
    int64_t ldaT;
    float *ac;
    int64_t ldac;
    int64_t M, F;
};

// 8 E4M3 codes -> fp32, times s (each code is exact in fp16, so the product is the
// one rounding).
__device__ __forceinline__ void decode8(uint2 c, float s, float (&f)[8])
{
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t two = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        f[2 * i] = lo * s;
        f[2 * i + 1] = hi * s;
    }
}

// A CTA takes a 128 x 128 tile of [M, F]; thread t rows 4 (t / 16) .. + 3 and columns
// 8 (t % 16) .. + 7, all in registers.  A row's 16 lanes are its 1x128 group; column
// maxima go over the rows of a thread, the two halves of a warp and, in shared memory,
// the 16 warps.
__global__ void __launch_bounds__(THREADS, 1) k_gate_bwd(const GateBwd p)
{
    pdl_begin();
    extern __shared__ __align__(16) uint8_t smem[];
    float *part = reinterpret_cast<float *>(smem + 3 * TILE_BYTES);  // [warp][3][128]
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4, warp = t >> 5;
    const int64_t m0 = (int64_t)blockIdx.x * GRP, f0 = (int64_t)blockIdx.y * GRP;
    const int rows = (int)(p.M - m0 < GRP ? p.M - m0 : GRP);
    const int64_t fb = p.F / GRP;  // scale rows of one projection
    uint4 va[4];
    uint2 vg[4], vu[4];
    float sg_[4], su_[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * rg + i;
        const bool in = r < rows;
        const int64_t m = m0 + r;
        const uint8_t *gp = p.guq + m * p.ldguq + f0 + 8 * cg;
        va[i] = in ? ld_stream(p.da + m * p.ldda + f0 + 8 * cg) : make_uint4(0, 0, 0, 0);
        vg[i] = in ? *reinterpret_cast<const uint2 *>(gp) : make_uint2(0, 0);
        vu[i] = in ? *reinterpret_cast<const uint2 *>(gp + p.F) : make_uint2(0, 0);
        sg_[i] = in ? p.gus[(int64_t)blockIdx.y * p.ld_gus + m] : 0.0f;
        su_[i] = in ? p.gus[(fb + blockIdx.y) * p.ld_gus + m] : 0.0f;
    }
    float dg[4][8], du[4][8], a[4][8], cmax[3][8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        cmax[0][j] = cmax[1][j] = cmax[2][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float g[8], u[8], d[8];
        decode8(vg[i], sg_[i], g);
        decode8(vu[i], su_[i], u);
        unpack8(va[i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sg = sigmoid_fast(g[j]);
            const float gs = g[j] * sg;
            du[i][j] = d[j] * gs;
            a[i][j] = gs * u[j];
            dg[i][j] = (d[j] * u[j]) * fmaf(gs, 1.0f - sg, sg);
            cmax[0][j] = fmaxf(cmax[0][j], fabsf(dg[i][j]));
            cmax[1][j] = fmaxf(cmax[1][j], fabsf(du[i][j]));
            cmax[2][j] = fmaxf(cmax[2][j], fabsf(a[i][j]));
        }
        const float s0 = group_scale(half_warp_max(max_abs8(dg[i])));
        const float s1 = group_scale(half_warp_max(max_abs8(du[i])));
        const int r = 4 * rg + i;
        if (r < rows) {
            const int64_t m = m0 + r;
            uint8_t *qp = p.q + m * p.ldq + f0 + 8 * cg;
            *reinterpret_cast<uint2 *>(qp) = encode8f(dg[i], s0, scale_rcp(s0));
            *reinterpret_cast<uint2 *>(qp + p.F) = encode8f(du[i], s1, scale_rcp(s1));
            if (cg == 0) {
                p.s[(int64_t)blockIdx.y * p.lds + m] = s0;
                p.s[(fb + blockIdx.y) * p.lds + m] = s1;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = fmaxf(cmax[k][j], __shfl_xor_sync(0xFFFFFFFFu, cmax[k][j], 16));
            if ((t & 16) == 0)
                part[(warp * 3 + k) * GRP + 8 * cg + j] = c;
        }
    __syncthreads();
    if (t < 3 * GRP) {
        float v = part[t];
#pragma unroll
        for (int w = 1; w < 16; ++w)
            v = fmaxf(v, part[w * 3 * GRP + t]);
        v = group_scale(v);
        part[t] = v;
        part[3 * GRP + t] = scale_rcp(v);
        const int k = t >> 7, c = t & 127;
        if (k < 2)
            p.sc[(int64_t)blockIdx.x * p.ldsc + k * p.F + f0 + c] = v;
        else
            p.ac[(int64_t)blockIdx.x * p.ldac + f0 + c] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * cg + j;
            const float s = part[k * GRP + c], r = part[(3 + k) * GRP + c];
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = k == 0 ? dg[i][j] : k == 1 ? du[i][j] : a[i][j];
                v[i] = r != 0.0f ? x * r : __fdiv_rn(x, s);
            }
            *reinterpret_cast<uint32_t *>(smem + k * TILE_BYTES + c * GRP + 8 * ((rg >> 1) ^ cg) + 4 * (rg & 1)) =
                e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16);
        }
    __syncthreads();
    store_tile_T(smem, t, THREADS, rows, p.qT + f0 * p.ldqT + m0, p.ldqT);
    store_tile_T(smem + TILE_BYTES, t, THREADS, rows, p.qT + (p.F + f0) * p.ldqT + m0, p.ldqT);
    store_tile_T(smem + 2 * TILE_BYTES, t, THREADS, rows, p.aT + f0 * p.ldaT + m0, p.ldaT);
}

}  // namespace

cudaError_t launch_gated_backward(const uint16_t *da, int64_t ldda, const uint8_t *guq, int64_t ldguq, const float *gus,
                                  int64_t ld_gus, uint8_t *q, int64_t ldq, float *s, int64_t lds, uint8_t *qT,
                                  int64_t ldqT, float *sc, int64_t ldsc, uint8_t *aT, int64_t ldaT, float *ac,
                                  int64_t ldac, int64_t M, int64_t F, cudaStream_t st)
{
    const GateBwd p = {da, ldda, guq, ldguq, gus, ld_gus, q,    ldq, s,    lds, qT,
                       ldqT, sc, ldsc, aT, ldaT, ac, ldac, M,  F};
    const cudaError_t e = cudaFuncSetAttribute(k_gate_bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(k_gate_bwd, dim3((unsigned)((M + GRP - 1) / GRP), (unsigned)(F / GRP)), dim3(THREADS), SMEM_BYTES,
                      st, p);
}

}  // namespace rlq
