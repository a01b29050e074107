// Element-level device helpers shared by the translation units of librlq.so:
// streaming loads, bf16 and E4M3 conversions, the scale rule of a group and the
// FP8 codes of fp32 values.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rlq {
namespace {

// Loads of a kernel's input, which no thread of the kernel writes: the read-only
// path without L1 allocation (measured 2% faster for the dual quantizer than an
// evict-first streaming load, the same elsewhere).
__device__ __forceinline__ uint4 ld_stream(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf_lo(w[i]);
        f[2 * i + 1] = bf_hi(w[i]);
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float2 v)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
    return d;
}

// Two E4M3 codes, RN-even with saturation to +-448: `lo` in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Scale of a group: fl32(amax / 448), 1 for an all-zero group.
__device__ __forceinline__ float group_scale(float amax)
{
    return amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f);
}

// Multiplier that turns x into x / s before the encoding: RN(1 / s).  The
// operators that quantize fp32 results use the product x * RN(1/s), at most
// 1.5 ulp from the quotient, where the values themselves carry as much.  Scales
// below 2^-100 (their reciprocal may overflow) return 0: encode8f divides then.
__device__ __forceinline__ float scale_rcp(float s) { return s < 0x1p-100f ? 0.0f : __frcp_rn(s); }

// E4M3 codes of 8 fp32 values of one group (scale s, rcp = scale_rcp(s)).
__device__ __forceinline__ uint2 encode8f(const float (&v)[8], float s, float rcp)
{
    float f[8];
    if (rcp != 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = v[i] * rcp;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __fdiv_rn(v[i], s);
    }
    return make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16),
                      e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
}

__device__ __forceinline__ float max_abs8(const float (&v)[8])
{
    const float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    const float b = fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7])));
    return fmaxf(a, b);
}

// 1 / (1 + exp(-g)) with the exponential and the reciprocal of the special-function
// units (about 2 and 1 ulp); 0 where exp(-g) overflows.
__device__ __forceinline__ float sigmoid_fast(float g)
{
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
    return r;
}

// Maximum over the 16 lanes of a half-warp (all 32 lanes take part).
__device__ __forceinline__ float half_warp_max(float a)
{
#pragma unroll
    for (int o = 8; o; o >>= 1)
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    return a;
}

// Writes a 128 x 128 tile of codes, held as [column][16 chunks of 8 rows] with chunk
// index XOR column / 8, as rows of the transposed matrix: 8 threads per column, 16
// bytes each.  Rows at or past `rows` are not written.  dst: element (column 0, row 0).
__device__ __forceinline__ void store_tile_T(const uint8_t *tile, int t, int threads, int rows,
                                             uint8_t *__restrict__ dst, int64_t ld)
{
    const int i = t & 7;
    for (int c = t >> 3; c < 128; c += threads >> 3) {
        const int cg = c >> 3;
        uint4 v = *reinterpret_cast<const uint4 *>(tile + c * 128 + 16 * (i ^ (cg >> 1)));
        if (cg & 1)
            v = make_uint4(v.z, v.w, v.x, v.y);
        uint8_t *p = dst + (int64_t)c * ld + 16 * i;
        if (16 * i + 16 <= rows) {
            *reinterpret_cast<uint4 *>(p) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int b = 0; b < 16; ++b)
                if (16 * i + b < rows)
                    p[b] = (uint8_t)(w[b >> 2] >> (8 * (b & 3)));
        }
    }
}

}  // namespace
}  // namespace rlq
