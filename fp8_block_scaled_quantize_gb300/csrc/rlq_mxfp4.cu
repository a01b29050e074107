// MXFP4 quantizer and dequantizer (sm_103a).
//
// OCP Microscaling Formats v1.0, MXFP4: blocks of 32 consecutive elements, E2M1 values and
// one E8M0 scale, a power of two.  With amax the block's largest magnitude,
//   e = clamp(floor(log2(amax)) - 2, -127, 127)  (-127 for a block of zeros)
//   q = E2M1_RNsat(x 2^-e),  scale byte e + 127  (255, a NaN, where the block holds an infinity or a NaN)
// 2 is the exponent of E2M1's largest value, 6.  x 2^-e is exact, so every code and scale is
// determined bit for bit; of a bf16 amax the byte is its exponent field less 2, at least 0.
//
// Scales lie in 512-byte tiles of 128 rows x 4 blocks, row tiles outer, byte
// (r % 32) 16 + (r % 128) / 32 4 + b % 4 of tile (r / 128, b / 4): the order in which
// tcgen05.cp takes 32 lanes x 16 bytes into tensor memory, so the product copies them as
// they are.  A warp therefore quantizes rows r, r + 32, r + 64 and r + 96 of a row tile, 128
// columns of each at a time: their 16 scale bytes are one piece.
//
// Bound by memory: 2 bytes a value read, 17/32 written, per direction.
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"

namespace rlq {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

// The largest magnitude's bits in each half of the words' 16-bit halves.
template <int N>
__device__ __forceinline__ uint32_t max_halves(const uint32_t (&w)[N])
{
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < N; ++i)
        m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return m;
}

// Scale byte of a block whose largest magnitude has the bf16 bits `amax`.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    const int f = (int)(amax >> 7);
    return f == 255 ? 255u : (uint32_t)max(f - 2, 0);
}

// 2^-e of a scale byte (255: any value, the scale itself is the NaN).
__device__ __forceinline__ float rcp_of(uint32_t s) { return __uint_as_float((254u - min(s, 253u)) << 23); }

// 2^e of a scale byte, a NaN for 255.
__device__ __forceinline__ float value_of(uint32_t s)
{
    return __uint_as_float(s == 255u ? 0x7FC00000u : s == 0u ? 0x00400000u : s << 23);
}

// E2M1 codes of eight values, the first in the lowest four bits: RN-even, saturating at
// +-6, the sign of zero kept (hardware conversion).
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&v)[4])
{
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d)
        : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    return d;
}

// Codes and scale byte of 8 of a row block's 32 values, the others in the three lanes
// beside this one (lanes 4 i .. 4 i + 3 hold a block).
__device__ __forceinline__ uint32_t row_codes(const uint4 &v, uint32_t *scale)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = max_halves(w);
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    *scale = scale_byte(max(m & 0xFFFFu, m >> 16));
    const float r = rcp_of(*scale);
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __fmul2_rn(make_float2(bf_lo(w[i]), bf_hi(w[i])), make_float2(r, r));
    return e2m1x8(f);
}

// The four scale bytes of a row's 128 columns (16 lanes, 4 to a block) as one word.
__device__ __forceinline__ uint32_t row_scales(uint32_t s, int lane)
{
    uint32_t w = s << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
    return w | __shfl_xor_sync(0xFFFFFFFFu, w, 8);
}

// Rows: a warp takes the four rows of a row tile that share 16 scale bytes, U column
// tiles of them, half a warp to a row: 16 bytes a lane and load, 2 U loads in flight.
template <int U>
__global__ void __launch_bounds__(THREADS)
    k_mx_rows(const uint16_t *__restrict__ x, int64_t M, int64_t K, int64_t ldx, uint8_t *__restrict__ q, int64_t ldq,
              uint8_t *__restrict__ s, int rv, int64_t items)
{
    pdl_begin();
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const int64_t id = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (id >= items)
        return;
    const int64_t ctiles = (K + 127) / 128, chunks = (ctiles + U - 1) / U;
    // (neighbouring warps: neighbouring rows, whose scale pieces are neighbours too)
    const int64_t rest = id / rv, rt = rest / chunks, ct0 = (rest - rt * chunks) * U;
    const int r = (int)(id - rest * rv);
    const int64_t row0 = rt * 128 + r + 32 * half;
    uint4 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = row0 + 64 * j, col = (ct0 + u) * 128 + l * 8;
            v[u][j] = row < M && col < K ? ld_stream(x + row * ldx + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t ct = ct0 + u;
        if (ct >= ctiles)
            break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t sb;
            const uint32_t codes = row_codes(v[u][j], &sb);
            const uint32_t sw = row_scales(sb, lane);
            const int64_t row = row0 + 64 * j, col = ct * 128 + l * 8;
            if (row < M) {
                if (col < K)
                    *reinterpret_cast<uint32_t *>(q + row * ldq + col / 2) = codes;
                if (l == 0)
                    *reinterpret_cast<uint32_t *>(s + (rt * ctiles + ct) * 512 + r * 16 + (half + 2 * j) * 4) = sw;
            }
        }
    }
}

// Rows and columns from one read: a CTA takes a 128 x 128 tile, quantizes its rows as
// above while it puts the values to shared memory, then its columns from there, two
// columns of 32 rows a thread (both halves of a word at once).  Row r of the tile lies at
// word 64 r + 8 (r / 32): the four row blocks that a warp reads fall into different banks.
__global__ void __launch_bounds__(THREADS)
    k_mx_both(const uint16_t *__restrict__ x, int64_t M, int64_t K, int64_t ldx, uint8_t *__restrict__ q, int64_t ldq,
              uint8_t *__restrict__ s, uint8_t *__restrict__ qT, int64_t ldqT, uint8_t *__restrict__ sT)
{
    pdl_begin();
    __shared__ __align__(16) uint32_t tile[128 * 64 + 3 * 8 + 8];
    __shared__ __align__(16) uint8_t col_scales[512];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, half = lane >> 4, l = lane & 15;
    const int64_t ctiles = (K + 127) / 128, rtiles = (M + 127) / 128;
    const int64_t rt = blockIdx.x / ctiles, ct = blockIdx.x - rt * ctiles;
    const int64_t col = ct * 128 + l * 8;
    uint4 v[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = rt * 128 + warp + 8 * i + 32 * half + 64 * j;
            v[i][j] = row < M && col < K ? ld_stream(x + row * ldx + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = warp + 8 * i, rb = half + 2 * j;  // row r + 32 rb of the tile
            const int64_t row = rt * 128 + r + 32 * rb;
            *reinterpret_cast<uint4 *>(&tile[(r + 32 * rb) * 64 + 8 * rb + 4 * l]) = v[i][j];
            uint32_t sb;
            const uint32_t codes = row_codes(v[i][j], &sb);
            const uint32_t sw = row_scales(sb, lane);
            if (row < M) {
                if (col < K)
                    *reinterpret_cast<uint32_t *>(q + row * ldq + col / 2) = codes;
                if (l == 0)
                    *reinterpret_cast<uint32_t *>(s + (rt * ctiles + ct) * 512 + r * 16 + rb * 4) = sw;
            }
        }
    __syncthreads();
    const int b = t & 3, cp = t >> 2;  // rows 32 b .., columns 2 cp and 2 cp + 1
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        w[i] = tile[(32 * b + i) * 64 + 8 * b + cp];
    const uint32_t m = max_halves(w);
    const int64_t off = rt * 64 + 16 * b, left = (M + 1) / 2 - off;  // bytes of the transposed row, and what it has from there
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sb = scale_byte(h ? m >> 16 : m & 0xFFFFu);
        const float rc = rcp_of(sb);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = w[8 * i + 2 * k], c = w[8 * i + 2 * k + 1];
                f[k] = __fmul2_rn(h ? make_float2(bf_hi(a), bf_hi(c)) : make_float2(bf_lo(a), bf_lo(c)),
                                  make_float2(rc, rc));
            }
            o[i] = e2m1x8(f);
        }
        const int c = 2 * cp + h;
        col_scales[(c & 31) * 16 + (c >> 5) * 4 + b] = (uint8_t)sb;
        if (ct * 128 + c < K && left > 0) {
            uint8_t *p = qT + (ct * 128 + c) * ldqT + off;
            const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
            if (left >= 16)
                *reinterpret_cast<uint4 *>(p) = o4;
            else
                store_head(p, o4, (int)left);
        }
    }
    __syncthreads();
    if (t < 32)
        *reinterpret_cast<uint4 *>(sT + (ct * rtiles + rt) * 512 + t * 16) =
            *reinterpret_cast<const uint4 *>(&col_scales[t * 16]);
}

// The n (1 .. 4) bytes that a row still has.
__device__ __forceinline__ uint32_t load_cut(const uint8_t *p, int n)
{
    uint32_t w = 0;
    for (int i = 0; i < n; ++i)
        w |= (uint32_t)p[i] << (8 * i);
    return w;
}

// Values of packed codes: the rows' kernel the other way round.  Every value is exact in bf16.
template <int U>
__global__ void __launch_bounds__(THREADS)
    k_mx_values(const uint8_t *__restrict__ q, int64_t ldq, const uint8_t *__restrict__ s, int64_t M, int64_t K,
                uint16_t *__restrict__ x, int64_t ldx, int rv, int64_t items)
{
    pdl_begin();
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const int64_t id = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (id >= items)
        return;
    const int64_t ctiles = (K + 127) / 128, chunks = (ctiles + U - 1) / U;
    const int64_t rest = id / rv, rt = rest / chunks, ct0 = (rest - rt * chunks) * U;
    const int r = (int)(id - rest * rv);
    const int64_t row0 = rt * 128 + r + 32 * half;
    uint32_t v[U][2];
    uint32_t sb[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = row0 + 64 * j, ct = ct0 + u, col = ct * 128 + l * 8;
            const bool in = row < M && col < K;
            v[u][j] = !in ? 0u
                      : col + 8 <= K ? __ldg(reinterpret_cast<const uint32_t *>(q + row * ldq + col / 2))
                                     : load_cut(q + row * ldq + col / 2, (int)(K - col + 1) / 2);
            sb[u][j] = in ? __ldg(s + (rt * ctiles + ct) * 512 + r * 16 + (half + 2 * j) * 4 + (l >> 2)) : 0u;
        }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = row0 + 64 * j, col = (ct0 + u) * 128 + l * 8;
            if (row >= M || col >= K)
                continue;
            uint32_t h[4];
            asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                "mov.b32 {a, b, c, d}, %4;\n\t"
                "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
                "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
                "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
                "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
                : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                : "r"(v[u][j]));
            const float sc = value_of(sb[u][j]);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                    : "=f"(lo), "=f"(hi)
                    : "r"(h[i]));
                o[i] = pack_bf16x2(__fmul2_rn(make_float2(lo, hi), make_float2(sc, sc)));
            }
            uint16_t *p = x + row * ldx + col;
            if (col + 8 <= K)
                *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
            else
                store_head(reinterpret_cast<uint8_t *>(p), make_uint4(o[0], o[1], o[2], o[3]), (int)(K - col) * 2);
        }
}

// Warps of a rows' kernel with U column tiles a warp: row tiles x chunks x the rows of a
// row tile's first 32 that exist.
int64_t row_items(int64_t M, int64_t K, int U, int *rv)
{
    const int64_t ctiles = (K + 127) / 128;
    *rv = M < 32 ? (int)M : 32;
    return (M + 127) / 128 * ((ctiles + U - 1) / U) * *rv;
}

}  // namespace

cudaError_t launch_quant_mxfp4(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, uint8_t *q, int64_t ldq, uint8_t *s,
                               uint8_t *qT, int64_t ldqT, uint8_t *sT, cudaStream_t st)
{
    if (qT)
        return launch_pdl(k_mx_both, dim3((unsigned)((M + 127) / 128 * ((K + 127) / 128))), dim3(THREADS), 0, st, x, M,
                          K, ldx, q, ldq, s, qT, ldqT, sT);
    int rv;
    int64_t items = row_items(M, K, 2, &rv);
    return launch_pdl(k_mx_rows<2>, dim3((unsigned)((items + WARPS - 1) / WARPS)), dim3(THREADS), 0, st, x, M, K, ldx, q,
                      ldq, s, rv, items);
}

cudaError_t launch_dequant_mxfp4(const uint8_t *q, int64_t ldq, const uint8_t *s, int64_t rows, int64_t cols,
                                 uint16_t *x, int64_t ldx, cudaStream_t st)
{
    int rv;
    const int64_t items = row_items(rows, cols, 2, &rv);
    return launch_pdl(k_mx_values<2>, dim3((unsigned)((items + WARPS - 1) / WARPS)), dim3(THREADS), 0, st, q, ldq, s, rows,
                      cols, x, ldx, rv, items);
}

}  // namespace rlq
