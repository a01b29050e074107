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
// Floor: 2 + 1 + 1 bytes read and 2 + 2 + 1 written per element of [M, F], 160 us at 8192
// x 14336 at the HBM rate.  Measured 198 us (0.81): instructions (decoding, the sigmoid,
// three maxima and five encodings an element, 35 in all), issued at 51% by the 16 warps a
// SM that the values' registers allow; a copy of the kernel without loads and stores was
// 15 us faster.  What brought it there from 294: the transposed codes
// stored as TMA boxes rather than by the threads (265 with 16-byte copies and bulk copies
// of single columns, 235 with boxes), the boxes' reads waited for a barrier later (223),
// inputs by TMA (211), two tiles ahead (203), scales without the
// IEEE division's and reciprocal's sequences (198).  Slower, each on top of the version of its
// time: all boxes from one warp (253 for 235), warps that store nothing running ahead of
// the boxes' issue (285), the row codes as boxes too (238), column maxima joined by 24
// lanes of every warp (248).  Earlier: the values formed twice at two CTAs a SM (303, 75
// instructions an element), pairs of half tiles that exchange row maxima across a cluster
// (335).
#include <cuda.h>
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"
#include "rlq_tc.cuh"

namespace rlq {
namespace {

constexpr int GRP = 128;
constexpr int THREADS = 512;
constexpr int LOADER = THREADS - 32;  // the thread that issues the input copies
// Shared memory: two tiles of input (da's 128 rows of 256 bytes, g's and u's codes) and their
// 2 x 128 scales, the three transposed code tiles, 16 warps' column maxima.
constexpr int IN_BYTES = 4 * GRP * GRP;
// A code tile is 128 slots of 128 bytes, a column's codes each: column 8 c + j in slot
// 16 j + c, its eight 16-byte chunks XOR c mod 8 (the 128-byte swizzle), so that the
// lanes that write one j differ in the bank.
constexpr int TILE_BYTES = GRP * GRP;
constexpr int OFF_SCALES = 2 * IN_BYTES;
constexpr int OFF_TILES = OFF_SCALES + 2 * 2 * GRP * 4;
constexpr int OFF_PART = OFF_TILES + 3 * TILE_BYTES;
constexpr int OFF_RCP = OFF_PART + 16 * 3 * GRP * 4;  // 3 x 128 reciprocals, 3 x 128 factors
constexpr int OFF_BARS = OFF_RCP + 2 * 3 * GRP * 4;  // two mbarriers, the abort flag
constexpr int SMEM_BYTES = OFF_BARS + 24;
static_assert(SMEM_BYTES <= 232448 && OFF_TILES % 1024 == 0, "shared memory budget; the swizzle's period");

struct GateBwd {
    const float *gus;  // (da and the checkpoint's codes come through tensor maps)
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
    int m_tiles, tiles;
    uint64_t timeout_ns;
    int withhold_first_load;  // diagnostic: nothing arrives for the CTA's first tile
};

// A barrier of the CTA that some warps wait at and others only pass.
__device__ __forceinline__ void bar_wait()
{
    asm volatile("bar.sync %0, %1;" ::"n"(1), "n"(THREADS) : "memory");
}
__device__ __forceinline__ void bar_pass()
{
    asm volatile("bar.arrive %0, %1;" ::"n"(1), "n"(THREADS) : "memory");
}
// Shared -> global by the copy engine: a box of 16 columns of 128 codes.
__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// 8 E4M3 codes -> fp32, times s (each code is exact in fp16, so the product is the
// one rounding).
__device__ __forceinline__ void decode8(uint2 c, float s, float2 (&f)[4])
{
    const uint32_t w[2] = {c.x, c.y};
    uint32_t h4[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(h4[2 * i]), "=r"(h4[2 * i + 1])
            : "r"(w[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = h4[i];
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        f[i] = __fmul2_rn(make_float2(lo, hi), make_float2(s, s));
    }
}

// Persistent, one CTA per SM, 128 x 128 tiles of [M, F], row block fastest.  Thread t
// has rows 4 (t / 16) .. + 3 and columns 8 (t % 16) .. + 7 of a tile, all of it in
// registers; the next two arrive in shared memory by TMA meanwhile.  A
// row's 16 lanes are its 1x128 group: the eight row maxima of a half-warp (four rows of
// dg, four of du) are reduced in one transposed exchange (each step hands half of the
// remaining ones to the partner lane), after which a lane pair holds one group's and
// computes its scale once.  Column maxima go over the rows of a thread, the two halves
// of a warp and, in shared memory, the 16 warps.
__global__ void __launch_bounds__(THREADS, 1) k_gate_bwd(const GateBwd p, const __grid_constant__ CUtensorMap tmQ,
                                                         const __grid_constant__ CUtensorMap tmA,
                                                         const __grid_constant__ CUtensorMap tmDa,
                                                         const __grid_constant__ CUtensorMap tmGu)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    float *part = reinterpret_cast<float *>(smem + OFF_PART);  // [warp][3][128]
    float *rcp = reinterpret_cast<float *>(smem + OFF_RCP);    // [3][128], factors behind them
    uint8_t *tiles = smem + OFF_TILES;
    const uint32_t smem0 = (uint32_t)__cvta_generic_to_shared(smem);
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4, warp = t >> 5;
    const bool b3 = t & 8, b2 = t & 4, b1 = t & 2;
    const int own = (t & 15) >> 1;  // the group maximum this lane ends up with: matrix own / 4, row own % 4
    const int64_t fb = p.F / GRP;   // scale rows of one projection

    // Row block and column block of a tile, and the step from one of this CTA's tiles to
    // the next.
    int mt = blockIdx.x % p.m_tiles, ft = blockIdx.x / p.m_tiles;
    const int step_m = gridDim.x % p.m_tiles, step_f = gridDim.x / p.m_tiles;
    const uint32_t bars = smem0 + OFF_BARS;
    volatile uint32_t *abort_flag = reinterpret_cast<uint32_t *>(smem + OFF_BARS + 16);
    if (t == LOADER) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        *abort_flag = 0;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        prefetch_tmap(&tmDa);
        prefetch_tmap(&tmGu);
    }
    __syncthreads();
    pdl_begin();
    auto prefetch = [&](int pm, int pf, int buf, bool inputs = true) {
        const int64_t m = (int64_t)pm * GRP + 4 * rg;
        const int left = (int)(p.M - m < 4 ? p.M - m : 4);  // rows of mine inside the matrix (may be <= 0)
        if (t == LOADER && inputs && !*abort_flag) {  // (rows past the end arrive as zeros)
            const uint32_t bar = bars + 8 * buf, in = smem0 + buf * IN_BYTES;
            mbar_arrive_expect_tx(bar, IN_BYTES);
            tma_load_2d(in, &tmDa, bar, pf * GRP, pm * GRP);
            tma_load_2d(in + 2 * GRP * GRP, &tmGu, bar, pf * GRP, pm * GRP);
            tma_load_2d(in + 3 * GRP * GRP, &tmGu, bar, (int)p.F + pf * GRP, pm * GRP);
        }
        if (cg < 8) {  // this half-warp's scales: four rows of g, four of u
            const bool ok = (cg & 3) < left;
            cp_async4(smem0 + OFF_SCALES + (buf * 2 * GRP + 8 * rg + cg) * 4,
                  ok ? p.gus + ((cg >> 2) * fb + pf) * p.ld_gus + m + (cg & 3) : p.gus, ok ? 4 : 0);
        }
    };

    auto step = [&](int &m, int &f) {
        m += step_m;
        f += step_f;
        if (m >= p.m_tiles) {
            m -= p.m_tiles;
            ++f;
        }
    };
    int tile = blockIdx.x, am = mt, af = ft;  // (am, af): the tile to copy next
    if (tile < p.tiles)
        prefetch(am, af, 0, !p.withhold_first_load);
    asm volatile("cp.async.commit_group;" ::: "memory");
    step(am, af);
    if (tile + (int)gridDim.x < p.tiles)
        prefetch(am, af, 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    step(am, af);
    for (uint32_t buf = 0, phase = 0; tile < p.tiles; tile += gridDim.x, phase ^= buf, buf ^= 1) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        // (Should the wait run out, this tile is formed from what is there, within the
        // buffers, the error word says so and the CTA leaves after it.)
        (void)mbar_wait(bars + 8 * buf, phase, abort_flag, p.timeout_ns, SITE_GATE_FULL);
        // A thread reads what its half-warp copied.  The last tile's codes may still be
        // leaving: shared memory that they use is written after the next barrier only.
        __syncwarp();
        const int64_t m0 = (int64_t)mt * GRP, f0 = (int64_t)ft * GRP;
        const int rows = (int)(p.M - m0 < GRP ? p.M - m0 : GRP);
        const uint8_t *in = smem + buf * IN_BYTES;
        const float *scl = reinterpret_cast<const float *>(smem + OFF_SCALES) + buf * 2 * GRP + 8 * rg;
        const float4 gs4 = *reinterpret_cast<const float4 *>(scl), us4 = *reinterpret_cast<const float4 *>(scl + 4);
        const float sg4[4] = {gs4.x, gs4.y, gs4.z, gs4.w}, su4[4] = {us4.x, us4.y, us4.z, us4.w};
        float2 val[3][4][4], cmax[3][4];  // dg, du, a of [row][column pair]
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 g[4], u[4];
            decode8(*reinterpret_cast<const uint2 *>(in + 2 * GRP * GRP + (4 * rg + i) * GRP + 8 * cg), sg4[i], g);
            decode8(*reinterpret_cast<const uint2 *>(in + 3 * GRP * GRP + (4 * rg + i) * GRP + 8 * cg), su4[i], u);
            const uint4 dv = *reinterpret_cast<const uint4 *>(in + (4 * rg + i) * 2 * GRP + 16 * cg);
            const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = make_float2(bf_lo(dw[j]), bf_hi(dw[j]));
                const float2 sg = sigmoid2(g[j]);
                const float2 gs = __fmul2_rn(g[j], sg);
                const float2 om = __ffma2_rn(sg, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
                val[0][i][j] = __fmul2_rn(__fmul2_rn(d, u[j]), __ffma2_rn(gs, om, sg));
                val[1][i][j] = __fmul2_rn(d, gs);
                val[2][i][j] = __fmul2_rn(gs, u[j]);
            }
            v[i] = max_abs8(val[0][i]);
            v[4 + i] = max_abs8(val[1][i]);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 m = make_float2(max3_abs(val[k][0][j].x, val[k][1][j].x, val[k][2][j].x),
                                             max3_abs(val[k][0][j].y, val[k][1][j].y, val[k][2][j].y));
                cmax[k][j] = make_float2(fmaxf(m.x, fabsf(val[k][3][j].x)), fmaxf(m.y, fabsf(val[k][3][j].y)));
            }
#pragma unroll
        for (int k = 0; k < 3; ++k)
            store_column_maxima(cmax[k], t & 16, part + (warp * 3 + k) * GRP + 8 * cg);
        float cs = 1.0f;
        if (t >= 3 * GRP) {
            bar_pass();
        } else {
            bar_wait();
            float c = part[t];
#pragma unroll
            for (int w = 1; w < 16; ++w)
                c = fmaxf(c, part[w * 3 * GRP + t]);
            cs = group_scale(c);
            const int k = t >> 7, cc = t & 127;
            if (k < 2)
                p.sc[(int64_t)mt * p.ldsc + k * p.F + f0 + cc] = cs;
            else
                p.ac[(int64_t)mt * p.ldac + f0 + cc] = cs;
            rcp[t] = scale_rcp(cs);
        }
        // row groups
        float x4[4], x2[2], x1;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x4[k] = fmaxf(b3 ? v[k + 4] : v[k], __shfl_xor_sync(0xFFFFFFFFu, b3 ? v[k] : v[k + 4], 8));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            x2[k] = fmaxf(b2 ? x4[k + 2] : x4[k], __shfl_xor_sync(0xFFFFFFFFu, b2 ? x4[k] : x4[k + 2], 4));
        x1 = fmaxf(b1 ? x2[1] : x2[0], __shfl_xor_sync(0xFFFFFFFFu, b1 ? x2[0] : x2[1], 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 1));
        const float rs = group_scale(x1), rr = scale_rcp(rs), rp = scale_pre(rs);
        if ((t & 1) == 0 && 4 * rg + (own & 3) < rows)
            p.s[((own >> 2) * fb + ft) * p.lds + m0 + 4 * rg + (own & 3)] = rs;
        uint8_t *qp = p.q + (m0 + 4 * rg) * p.ldq + f0 + 8 * cg;
        const int left = rows - 4 * rg;
        if (__any_sync(0xFFFFFFFFu, rp != 1.0f)) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = k & 3, src = (t & 16) + 2 * k;
                const float q = __shfl_sync(0xFFFFFFFFu, rr, src), pre = __shfl_sync(0xFFFFFFFFu, rp, src);
                if (i < left)
                    *reinterpret_cast<uint2 *>(qp + i * p.ldq + (k >> 2) * p.F) = encode8f(val[k >> 2][i], pre, q);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i, qp += p.ldq) {
                const float qg = __shfl_sync(0xFFFFFFFFu, rr, (t & 16) + 2 * i);
                const float qu = __shfl_sync(0xFFFFFFFFu, rr, (t & 16) + 8 + 2 * i);
                const uint2 cg8 = encode8f(val[0][i], 1.0f, qg), cu8 = encode8f(val[1][i], 1.0f, qu);
                if (i < left) {
                    *reinterpret_cast<uint2 *>(qp) = cg8;
                    *reinterpret_cast<uint2 *>(qp + p.F) = cu8;
                }
            }
        }
        // (the copies of the last tile's codes have read them: waited for by their issuers)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        // Column groups.  (Columns whose scale is below 2^-100 are scaled up first.)
        const int tiny = __syncthreads_or(cs < 0x1p-100f);
        // every thread has this tile's values: its buffer takes the one after the next
        if (tile + 2 * (int)gridDim.x < p.tiles)
            prefetch(am, af, buf);
        asm volatile("cp.async.commit_group;" ::: "memory");
        step(am, af);
        if (tiny) {
            if (t < 3 * GRP)
                rcp[3 * GRP + t] = scale_pre(cs);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = *reinterpret_cast<const float2 *>(rcp + (3 + k) * GRP + 8 * cg + 2 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        val[k][i][j] = __fmul2_rn(val[k][i][j], f);
                }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float4 r0 = *reinterpret_cast<const float4 *>(rcp + k * GRP + 8 * cg);
            const float4 r1 = *reinterpret_cast<const float4 *>(rcp + k * GRP + 8 * cg + 4);
            const float2 r[4] = {make_float2(r0.x, r0.y), make_float2(r0.z, r0.w), make_float2(r1.x, r1.y),
                                 make_float2(r1.z, r1.w)};
            uint8_t *out = tiles + k * TILE_BYTES + cg * GRP + 16 * ((rg >> 2) ^ (cg & 7)) + 4 * (rg & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = __fmul2_rn(val[k][i][j], r[j]);
                *reinterpret_cast<uint32_t *>(out + 2 * j * 16 * GRP) =
                    e4m3x4(y[0].x, y[1].x, y[2].x, y[3].x);
                *reinterpret_cast<uint32_t *>(out + (2 * j + 1) * 16 * GRP) =
                    e4m3x4(y[0].y, y[1].y, y[2].y, y[3].y);
            }
        }
        // The column codes leave by the copy engine, which reads shared memory through the
        // async proxy: 24 boxes, one or two a warp (all of them from one warp: 253 us at
        // the size above).  The last row block's by 16-byte and byte stores.
        // (raised before the last barrier or after the next one only: all threads agree)
        const bool stop = *abort_flag != 0;
        if (rows == GRP) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            const int b = warp + 16 * (t & 31);
            if (b < 24) {
                const int k = b >> 3, j = b & 7;
                store_box(k < 2 ? &tmQ : &tmA, smem0 + OFF_TILES + k * TILE_BYTES + j * 16 * GRP, (int)m0, j,
                          (int)(((k == 1 ? p.F : 0) + f0) >> 3));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        } else {
            __syncthreads();
            for (int b = t; b < 3 * GRP * 8; b += THREADS) {
                const int k = b >> 10, slot = (b >> 3) & 127, i = b & 7;
                const int64_t col = f0 + 8 * (slot & 15) + (slot >> 4);
                const uint4 c = *reinterpret_cast<const uint4 *>(tiles + k * TILE_BYTES + slot * GRP +
                                                                 16 * (i ^ (slot & 7)));
                uint8_t *dst = (k < 2 ? p.qT + (k * p.F + col) * p.ldqT : p.aT + col * p.ldaT) + m0 + 16 * i;
                if (16 * i + 16 <= rows)
                    *reinterpret_cast<uint4 *>(dst) = c;
                else if (16 * i < rows)
                    store_head(dst, c, rows - 16 * i);
            }
        }
        if (stop) {
            if (t == LOADER) {  // copies still in flight land before the CTA's memory is given up
                uint32_t never = 0;
                mbar_wait(bars + 8 * buf, phase, &never, 20000000ull, SITE_DRAIN);
                if (tile + (int)gridDim.x < p.tiles)
                    mbar_wait(bars + 8 * (buf ^ 1), phase ^ buf, &never, 20000000ull, SITE_DRAIN);
            }
            break;
        }
        step(mt, ft);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

rlq_status launch_gated_backward(const uint16_t *da, int64_t ldda, const uint8_t *guq, int64_t ldguq, const float *gus,
                                  int64_t ld_gus, uint8_t *q, int64_t ldq, float *s, int64_t lds, uint8_t *qT,
                                  int64_t ldqT, float *sc, int64_t ldsc, uint8_t *aT, int64_t ldaT, float *ac,
                                  int64_t ldac, int64_t M, int64_t F, cudaStream_t st)
{
    const int64_t m_tiles = (M + GRP - 1) / GRP, tiles = m_tiles * (F / GRP);
    const GateBwd p = {gus,  ld_gus, q,    ldq, s, lds,          qT,         ldqT,           sc, ldsc, aT,
                       ldaT, ac,     ldac, M,   F, (int)m_tiles, (int)tiles, wait_limit_ns(),
                       take_stall() ? 1 : 0};
    CUtensorMap tmQ = {}, tmA = {}, tmDa, tmGu;
    rlq_status rin = encode_tile_map(&tmDa, da, true, M, F, ldda);
    if (rin == RLQ_OK)
        rin = encode_tile_map(&tmGu, guq, false, M, 2 * F, ldguq);
    if (rin != RLQ_OK)
        return rin;
    if (M >= GRP) {  // (a tile of fewer rows does without)
        rlq_status r = encode_columns_map(&tmQ, qT, M, 2 * F, ldqT);
        if (r == RLQ_OK)
            r = encode_columns_map(&tmA, aT, M, F, ldaT);
        if (r != RLQ_OK)
            return r;
    }
    // (once per device)
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !set[dev & 63].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(k_gate_bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        set[dev & 63].store(e == cudaSuccess, std::memory_order_relaxed);
    }
    if (e == cudaSuccess) {
        const int64_t sms = device_sms();
        e = launch_pdl(k_gate_bwd, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(THREADS), SMEM_BYTES, st, p, tmQ, tmA,
                       tmDa, tmGu);
    }
    return cuda_status(e, "gated backward launch");
}

cudaError_t take_gate_error_word(cudaStream_t st, unsigned long long *word) { return take_error_word(st, word); }

}  // namespace rlq
