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

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight E2M1 codes (one 32-bit word, element 0 in the lowest nibble) times one
// bf16 scale (in both halves of s2): four bf16x2 words, element 0 lowest.
// Magnitude bytes of 0, 0.5, 1, 1.5, 2, 3, 4, 6 in bf16: high bytes 00 3F 3F 3F 40
// 40 40 40, low bytes 00 00 80 C0 00 40 80 C0.  Signs: element 2k's sign is bit 7
// of byte k of (w << 4), element 2k+1's bit 7 of byte k of w; a prmt selector with
// bit 3 set replicates the selected byte's bit 7, so one prmt gives the sign bytes
// of four elements, which are merged into their high bytes before the interleave.
__device__ __forceinline__ uint4 e2m1x8_to_bf16(uint32_t w, uint32_t s2)
{
    constexpr uint32_t HI0 = 0x3F3F3F00u, HI1 = 0x40404040u;
    constexpr uint32_t LO0 = 0xC0800000u, LO1 = 0xC0804000u;
    const uint32_t m = w & 0x77777777u;  // magnitudes: prmt selectors in plain (not sign) mode
    const uint32_t m2 = m >> 16;
    const uint32_t we = w << 4;
    const uint32_t s03 = prmt(we, w, 0xD9C8u);  // signs of elements 0, 1, 2, 3 as 00 / FF bytes
    const uint32_t s47 = prmt(we, w, 0xFBEAu);  // elements 4 .. 7
    const uint32_t h03 = prmt(HI0, HI1, m) | (s03 & 0x80808080u);
    const uint32_t h47 = prmt(HI0, HI1, m2) | (s47 & 0x80808080u);
    const uint32_t l03 = prmt(LO0, LO1, m), l47 = prmt(LO0, LO1, m2);
    uint4 out;
    out.x = mul_bf16x2(prmt(l03, h03, 0x5140u), s2);  // elements 0, 1
    out.y = mul_bf16x2(prmt(l03, h03, 0x7362u), s2);  // elements 2, 3
    out.z = mul_bf16x2(prmt(l47, h47, 0x5140u), s2);
    out.w = mul_bf16x2(prmt(l47, h47, 0x7362u), s2);
    return out;
}

// Two E4M3 codes, RN-even with saturation to +-448: `lo` in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Four of them in a word, `a` in bits 0..7.  (One block of assembly, so that the pairs
// meet in the word without being widened first.)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// Scale of a group: fl32(amax / 448), 1 for an all-zero group, and 2^-149 where the quotient
// rounds to zero (amax <= 448 x 2^-150, which no bf16 value is but a product may be: codes
// by a scale of 0 would be NaN where the value is 0).  The quotient by
// Markstein's correction (IBM J. Res. Dev. 34(1), 1990): q = amax RN(1/448), then q +
// (amax - 448 q) RN(1/448), the remainder exact.  It was compared with the IEEE division
// for every finite amax >= 2^-117, where the quotient is normal, without a difference;
// the others divide.
__device__ __forceinline__ float group_scale(float amax)
{
    if (__float_as_uint(amax) - 0x05000000u < 0x7F800000u - 0x05000000u) {
        const float r = 1.0f / 448.0f, q = __fmul_rn(amax, r);
        return __fmaf_rn(__fmaf_rn(-q, 448.0f, amax), r, q);
    }
    // (the larger of the quotient's bits and 1: 2^-149 for 0)
    return amax == 0.0f ? 1.0f : __uint_as_float(max(__float_as_uint(__fdiv_rn(amax, 448.0f)), 1u));
}

// A scale as the encoding applies it: codes are of (x * pre) * rcp, with pre = 1, or
// 2^64 (exact) for scales below 2^-100, whose own reciprocal may overflow, and rcp =
// RN(1 / (s * pre)).  The operators that quantize fp32 results use this product, at
// most 1.5 ulp from the quotient x / s, where the values themselves carry as much.
__device__ __forceinline__ float scale_pre(float s) { return s < 0x1p-100f ? 0x1p64f : 1.0f; }
// One Newton step on the approximate reciprocal: correctly rounded for every s * pre that a
// finite amax gives (2^-100 to 2^120, each compared with __frcp_rn); zero, infinity and
// NaN keep the approximation's infinity, zero and NaN.
__device__ __forceinline__ float scale_rcp(float s)
{
    const float d = s * scale_pre(s);
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
    const float e = __fmaf_rn(-d, y, 1.0f);
    return e == e ? __fmaf_rn(e, y, y) : y;
}

// E4M3 codes of 8 fp32 values (adjacent pairs) of one group.
__device__ __forceinline__ uint2 encode8f(const float2 (&v)[4], float pre, float rcp)
{
    const float2 r2 = make_float2(rcp, rcp);
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = v[i];
    if (pre != 1.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __fmul2_rn(f[i], make_float2(pre, pre));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __fmul2_rn(f[i], r2);
    return make_uint2(e4m3x4(f[0].x, f[0].y, f[1].x, f[1].y),
                      e4m3x4(f[2].x, f[2].y, f[3].x, f[3].y));
}

// max(|a|, |b|, |c|) in one instruction.
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float max_abs8(const float2 (&v)[4])
{
    const float a = max3_abs(v[0].x, v[0].y, v[1].x), b = max3_abs(v[1].y, v[2].x, v[2].y);
    return max3_abs(max3_abs(a, v[3].x, v[3].y), b, b);
}

// 1 / (1 + exp(-g)) of two values, the exponential and the reciprocal on the
// special-function units (about 2 and 1 ulp).  Their .ftz forms, a single instruction
// each: exp(-g) below 2^-126 adds nothing to 1, and a sigmoid below 2^-126 is 0.
__device__ __forceinline__ float2 sigmoid2(float2 g)
{
    float2 d, r;
    const float2 e = __fmul2_rn(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d.x) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d.y) : "f"(e.y));
    d = __fadd2_rn(d, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
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

// The maxima of a thread's eight columns over its rows -> over both halves of the warp
// (lanes l and l ^ 16 hold the same columns), to eight consecutive floats at dst: the
// lower half keeps columns 0-3, the upper 4-7.
__device__ __forceinline__ void store_column_maxima(const float2 (&c)[4], bool upper, float *dst)
{
    float4 o;
    float *f = &o.x;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 keep = upper ? c[2 + j] : c[j], send = upper ? c[j] : c[2 + j];
        f[2 * j] = fmaxf(keep.x, __shfl_xor_sync(0xFFFFFFFFu, send.x, 16));
        f[2 * j + 1] = fmaxf(keep.y, __shfl_xor_sync(0xFFFFFFFFu, send.y, 16));
    }
    *reinterpret_cast<float4 *>(dst + (upper ? 4 : 0)) = o;
}

// The first n bytes (0 .. 15) of a 16-byte piece, p on a 16-byte boundary.
__device__ __forceinline__ void store_head(uint8_t *p, uint4 v, int n)
{
    if (n & 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(v.x, v.y);
        v.x = v.z;
        v.y = v.w;
        p += 8;
    }
    if (n & 4) {
        *reinterpret_cast<uint32_t *>(p) = v.x;
        v.x = v.y;
        p += 4;
    }
    if (n & 2) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)v.x;
        v.x >>= 16;
        p += 2;
    }
    if (n & 1)
        *p = (uint8_t)v.x;
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
        if (16 * i + 16 <= rows)
            *reinterpret_cast<uint4 *>(p) = v;
        else if (16 * i < rows)
            store_head(p, v, rows - 16 * i);
    }
}

}  // namespace
}  // namespace rlq
