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
// Bound by memory (2 bytes a value read once, 17/32 written per direction) where there is enough
// of it: rows of 8192 x 14336 in 48.4 us (0.90 of HBM), both ways 14336 x 4096 in 30.3 (0.87;
// the phases of a tile), read back 25.7 (0.85).  Small ones are bound by launch and load latency
// (333 x 18944: 4.5 us, 1 x 4096: 1.5).
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"

namespace rlq {
namespace {

// Rows' kernels, 1001 x 18944, written and read back: 17.8 us; 18.3 in CTAs of 256, 22.1 of 64.
constexpr int THREADS = 128, WARPS = THREADS / 32;
constexpr int BOTH_THREADS = 256, BOTH_CTAS_SM = 5;

// 16-byte global -> shared copy; src_bytes = 0 writes zeros.
__device__ __forceinline__ void cp_async16_zfill(void *dst, const void *src, uint32_t src_bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(src_bytes)
                 : "memory");
}

// The larger magnitude in each half of two bf16 pairs, with a sign that means nothing; a NaN if
// either is one.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b)
{
    uint32_t m;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

template <int N>
__device__ __forceinline__ uint32_t max_halves(const uint32_t (&w)[N])
{
    uint32_t m[4] = {w[0], w[1], w[2], w[3]};  // (four chains: N is 4, 16 or 32)
#pragma unroll
    for (int i = 4; i < N; ++i)
        m[i & 3] = max_abs2(m[i & 3], w[i]);
    return max_abs2(max_abs2(m[0], m[1]), max_abs2(m[2], m[3]));
}

// Scale byte of a block whose largest magnitude has the bf16 bits `amax`.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    const int f = (int)(amax >> 7);
    return f == 255 ? 255u : (uint32_t)max(f - 2, 0);
}

// 2^-e of a scale byte (255: any value, the scale itself is the NaN).
__device__ __forceinline__ float rcp_of(uint32_t s) { return __uint_as_float((254u - min(s, 253u)) << 23); }

// 2^e of a scale byte in bf16, twice; NaNs for 255.
__device__ __forceinline__ uint32_t value2_of(uint32_t s)
{
    const uint32_t b = s == 255u ? 0x7FC0u : s == 0u ? 0x0040u : s << 7;
    return b | (b << 16);
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
    m = max_abs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max_abs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    *scale = scale_byte(max(m & 0x7FFFu, m >> 16 & 0x7FFFu));
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

// What a warp of the rows' kernels works on: the four rows of a row tile that share 16 scale
// bytes, U column tiles of them, half a warp to a row: 16 bytes of values a lane and tile.
struct RowItem {
    int64_t row, rt, ct0, ctiles;  // this lane's first row (the other: row + 64), the tiles
    int r, l, half;
    int left;     // columns from this lane's first one, at most those of the U tiles
    bool in[2];   // the rows exist
    bool whole;   // nothing of the warp's is cut
};

template <int U>
__device__ __forceinline__ RowItem row_item(uint32_t id, int64_t M, int64_t K, uint32_t rv)
{
    RowItem it;
    const int lane = threadIdx.x & 31;
    it.half = lane >> 4;
    it.l = lane & 15;
    it.ctiles = (K + 127) / 128;
    const uint32_t chunks = (uint32_t)(it.ctiles + U - 1) / U;
    // (neighbouring warps: neighbouring rows, whose scale pieces are neighbours too)
    const uint32_t rest = id / rv, rt = rest / chunks;
    it.r = (int)(id - rest * rv);
    it.rt = rt;
    it.ct0 = (int64_t)(rest - rt * chunks) * U;
    it.row = it.rt * 128 + it.r + 32 * it.half;
    it.in[0] = it.row < M;
    it.in[1] = it.row + 64 < M;
    it.left = (int)min(K - it.ct0 * 128, (int64_t)(U * 128)) - it.l * 8;
    it.whole = __all_sync(0xFFFFFFFFu, it.in[1] && it.left + it.l * 8 == U * 128);
    return it;
}

template <int U, bool kEdge>
__device__ __forceinline__ void quantize_rows(const RowItem &it, const uint16_t *__restrict__ x, int64_t ldx,
                                              uint8_t *__restrict__ q, int64_t ldq, uint8_t *__restrict__ s)
{
    const uint16_t *const first = x;
    x += it.row * ldx + it.ct0 * 128 + it.l * 8;
    q += it.row * ldq + it.ct0 * 64 + it.l * 4;
    s += (it.rt * it.ctiles + it.ct0) * 512 + it.r * 16 + it.half * 4;
    uint4 v[U][2];
    // (what is cut reads the matrix's first values, so that all loads are in flight together)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            v[u][j] = ld_stream(!kEdge || (it.in[j] && 128 * u < it.left) ? x + 64 * j * ldx + 128 * u : first);
    if (kEdge) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (!(it.in[j] && 128 * u < it.left))
                    v[u][j] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t sb;
            const uint32_t codes = row_codes(v[u][j], &sb);
            const uint32_t sw = row_scales(sb, threadIdx.x & 31);
            if (!kEdge || (it.in[j] && 128 * u < it.left))
                *reinterpret_cast<uint32_t *>(q + 64 * j * ldq + 64 * u) = codes;
            if (it.l == 0 && (!kEdge || (it.in[j] && it.ct0 + u < it.ctiles)))
                *reinterpret_cast<uint32_t *>(s + 512 * u + 8 * j) = sw;
        }
}

template <int U>
__global__ void __launch_bounds__(THREADS)
    k_mx_rows(const uint16_t *__restrict__ x, int64_t M, int64_t K, int64_t ldx, uint8_t *__restrict__ q, int64_t ldq,
              uint8_t *__restrict__ s, uint32_t rv, uint32_t items)
{
    pdl_begin();
    const uint32_t id = blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (id >= items)
        return;
    const RowItem it = row_item<U>(id, M, K, rv);
    if (it.whole)
        quantize_rows<U, false>(it, x, ldx, q, ldq, s);
    else
        quantize_rows<U, true>(it, x, ldx, q, ldq, s);
}

// Rows and columns from one read: a CTA copies a 128 x 128 tile to shared memory, quantizes its
// rows from there, a block a thread and turn, and its columns, two columns of 32 rows a thread
// (both halves of a word at once).  Row r of the tile lies at word 68 r + 8 (r / 32): eight lanes'
// 16-byte reads of four rows' neighbouring blocks, and the words that a warp reads of four row
// blocks, fall into different banks.  (Rows as above, straight from their registers, with four lanes
// to a block, took 33.1 us for 14336 x 4096, this 30.3.)
struct BothArgs {
    const uint16_t *x;
    int64_t M, K, ldx;
    uint8_t *q;
    int64_t ldq;
    uint8_t *s, *qT;
    int64_t ldqT;
    uint8_t *sT;
    int ctiles, rtiles;
};

__device__ __forceinline__ int tile_word(int r) { return 68 * r + 8 * (r >> 5); }

// kEdge: the tile is cut by the matrix's end.
template <bool kEdge>
__device__ __forceinline__ void both_tile(const BothArgs &p, uint32_t *tile, uint8_t *row_scale, uint8_t *col_scale)
{
    const int t = threadIdx.x;
    const int rt = blockIdx.x / p.ctiles, ct = blockIdx.x - rt * p.ctiles;
    const int rows = kEdge ? (int)min(p.M - (int64_t)rt * 128, (int64_t)128) : 128;
    const int cols = kEdge ? (int)min(p.K - (int64_t)ct * 128, (int64_t)128) : 128;
    {
        const int l = t & 15, r0 = t >> 4;
        const uint16_t *x = p.x + ((int64_t)rt * 128 + r0) * p.ldx + ct * 128 + l * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = !kEdge || (r0 + 16 * i < rows && l * 8 < cols);
            cp_async16_zfill(tile + tile_word(r0 + 16 * i) + 4 * l, in ? x + (int64_t)16 * i * p.ldx : p.x, in ? 16u : 0u);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();
    {
        const int b = (t >> 2) & 3;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = (t & 3) + 4 * ((t >> 4) + 16 * k);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4 *>(w + 4 * i) = *reinterpret_cast<const uint4 *>(tile + tile_word(r) + 16 * b + 4 * i);
            const uint32_t m = max_halves(w);
            const uint32_t sb = scale_byte(max(m & 0x7FFFu, m >> 16 & 0x7FFFu));
            const float rc = rcp_of(sb);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[j] = __fmul2_rn(make_float2(bf_lo(w[4 * i + j]), bf_hi(w[4 * i + j])), make_float2(rc, rc));
                o[i] = e2m1x8(f);
            }
            row_scale[(r & 31) * 16 + (r >> 5) * 4 + b] = (uint8_t)sb;
            // (32 columns are a block's: K % 32 == 0)
            if (!kEdge || (r < rows && 32 * b < cols))
                *reinterpret_cast<uint4 *>(p.q + ((int64_t)rt * 128 + r) * p.ldq + ct * 64 + 16 * b) =
                    make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    const int b = t & 3, cp = t >> 2;  // rows 32 b .., columns 2 cp and 2 cp + 1
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        w[i] = tile[tile_word(32 * b) + 68 * i + cp];
    const uint32_t m = max_halves(w);
    const int left = (rows + 1) / 2 - 16 * b;  // bytes that the transposed row has of the thread's 16
    uint8_t *qT = p.qT + ((int64_t)ct * 128 + 2 * cp) * p.ldqT + rt * 64 + 16 * b;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sb = scale_byte((h ? m >> 16 : m) & 0x7FFFu);
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
        col_scale[(c & 31) * 16 + (c >> 5) * 4 + b] = (uint8_t)sb;
        if (!kEdge || (c < cols && left > 0)) {
            const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
            if (!kEdge || left >= 16)
                *reinterpret_cast<uint4 *>(qT + h * p.ldqT) = o4;
            else
                store_head(qT + h * p.ldqT, o4, left);
        }
    }
    __syncthreads();
    if (t < 64) {
        uint8_t *to = t < 32 ? p.s + ((int64_t)rt * p.ctiles + ct) * 512 : p.sT + ((int64_t)ct * p.rtiles + rt) * 512;
        const uint8_t *from = t < 32 ? row_scale : col_scale;
        *reinterpret_cast<uint4 *>(to + (t & 31) * 16) = *reinterpret_cast<const uint4 *>(from + (t & 31) * 16);
    }
}

__global__ void __launch_bounds__(BOTH_THREADS, BOTH_CTAS_SM) k_mx_both(const BothArgs p)
{
    pdl_begin();
    __shared__ __align__(16) uint32_t tile[128 * 68 + 3 * 8];
    __shared__ __align__(16) uint8_t row_scale[512], col_scale[512];
    const int rt = blockIdx.x / p.ctiles, ct = blockIdx.x - rt * p.ctiles;
    if ((int64_t)(rt + 1) * 128 <= p.M && (int64_t)(ct + 1) * 128 <= p.K)
        both_tile<false>(p, tile, row_scale, col_scale);
    else
        both_tile<true>(p, tile, row_scale, col_scale);
}

// The n (1 .. 4) bytes that a row still has.
__device__ __forceinline__ uint32_t load_cut(const uint8_t *p, int n)
{
    uint32_t w = 0;
    for (int i = 0; i < n; ++i)
        w |= (uint32_t)p[i] << (8 * i);
    return w;
}

// Values of packed codes: the rows' kernel the other way round.  Every value is exact in bf16, and
// so is the product of a code's magnitude and its power of two there.
template <int U, bool kEdge>
__device__ __forceinline__ void row_values(const RowItem &it, const uint8_t *__restrict__ q, int64_t ldq,
                                           const uint8_t *__restrict__ s, uint16_t *__restrict__ x, int64_t ldx)
{
    x += it.row * ldx + it.ct0 * 128 + it.l * 8;
    q += it.row * ldq + it.ct0 * 64 + it.l * 4;
    s += (it.rt * it.ctiles + it.ct0) * 512 + it.r * 16 + it.half * 4 + (it.l >> 2);
    uint32_t v[U][2], sb[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = it.left - 128 * u;
            const uint8_t *p = q + 64 * j * ldq + 64 * u;
            const bool in = !kEdge || (it.in[j] && n > 0);
            v[u][j] = !in ? 0u : !kEdge || n >= 8 ? __ldg(reinterpret_cast<const uint32_t *>(p)) : load_cut(p, (n + 1) / 2);
            sb[u][j] = in ? __ldg(s + 512 * u + 8 * j) : 0u;
        }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = it.left - 128 * u;
            const uint4 o = e2m1x8_to_bf16(v[u][j], value2_of(sb[u][j]));
            uint16_t *p = x + 64 * j * ldx + 128 * u;
            if (!kEdge || (it.in[j] && n >= 8))
                *reinterpret_cast<uint4 *>(p) = o;
            else if (it.in[j] && n > 0)
                store_head(reinterpret_cast<uint8_t *>(p), o, n * 2);
        }
}

template <int U>
__global__ void __launch_bounds__(THREADS)
    k_mx_values(const uint8_t *__restrict__ q, int64_t ldq, const uint8_t *__restrict__ s, int64_t M, int64_t K,
                uint16_t *__restrict__ x, int64_t ldx, uint32_t rv, uint32_t items)
{
    pdl_begin();
    const uint32_t id = blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (id >= items)
        return;
    const RowItem it = row_item<U>(id, M, K, rv);
    if (it.whole)
        row_values<U, false>(it, q, ldq, s, x, ldx);
    else
        row_values<U, true>(it, q, ldq, s, x, ldx);
}

// Warps of a rows' kernel with U column tiles a warp: row tiles x chunks x the rows of a
// row tile's first 32 that exist.  (Below 2^32 for every matrix below 2^41 values.)
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
    if (qT) {
        const BothArgs p = {x, M, K, ldx, q, ldq, s, qT, ldqT, sT, (int)((K + 127) / 128), (int)((M + 127) / 128)};
        return launch_pdl(k_mx_both, dim3((unsigned)((int64_t)p.ctiles * p.rtiles)), dim3(BOTH_THREADS), 0, st, p);
    }
    // Four column tiles a warp where they make a full wave of warps, else two (8192 x 14336: 48.2
    // and 51.6 us; 333 x 18944: 6.1 and 4.6).
    int rv;
    int64_t items = row_items(M, K, 4, &rv);
    const bool four = items >= (int64_t)64 * device_sms();
    if (!four)
        items = row_items(M, K, 2, &rv);
    return launch_pdl(four ? k_mx_rows<4> : k_mx_rows<2>, dim3((unsigned)((items + WARPS - 1) / WARPS)), dim3(THREADS), 0, st,
                      x, M, K, ldx, q, ldq, s, rv, items);
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
