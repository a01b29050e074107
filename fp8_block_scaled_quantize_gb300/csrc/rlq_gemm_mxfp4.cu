// MXFP4 x MXFP4 product on 5th-generation tensor cores (sm_103a).
//
//   Y[m, n] = sum_k x[m, k] w[n, k],   x = e2m1(code) 2^e, one e per 32 elements of K, w alike
//
// tcgen05.mma kind::mxf4 multiplies packed E2M1 operands and applies both operands' E8M0
// scales (two per row and instruction of K = 64) before it adds in fp32: a product of two
// 4-bit values and two powers of two is exact, so only the additions round.
//
// Roles (320 threads): warp 0 copies ahead by TMA, per stage of 256 contraction elements (128
// bytes a row) both operands' codes (128-byte swizzle) and their scale tiles as they lie in
// memory; warp 1 copies the stage's scales to tensor memory (tcgen05.cp, 512 bytes per 128 rows
// and 128 elements; tcgen05.cp and tcgen05.mma of one thread run in order) and issues four MMAs;
// warps 2-9, two groups of four, read the finished sums and store them.  Warps 0 and 1 stay
// converged and elect the lane that issues: from a thread of its own every copy and MMA
// took its operands to uniform registers first, and 8192 x 14336 x 4096 247 us instead of 143.
//   * Pairs (kPair): two CTAs, 256 rows of A x up to 256 of B (cta_group::2), persistent.  The tokens
//     are A, so a lane holds neighbouring outputs of one token, which go to a swizzled box of
//     its warp's in shared memory by 16-byte stores and leave by TMA (the lanes of a column
//     apart, and swapped pairs, had 18944 x 3584 x 1001 take 88 and 44 us; it takes 35).  Where y's rows
//     are not on 16-byte boundaries, the weights are A, and a lane stores its column of y.
//     Two accumulators of 256 columns and the scales do not fit the 512 columns of tensor
//     memory, so the second one begins 32 columns before the first one's end; the epilogue reads
//     those columns first, and the next tile's MMAs start behind that.
//   * Single CTAs: 128 weight rows as A, the tokens as B: a few tokens are a narrow MMA, and a
//     store of 32 lanes is 32 neighbouring outputs of a token.  Where there are too few tiles for the
//     SMs, a cluster of up to 8 CTAs shares a tile's contraction; each CTA sends its part, 16 bytes
//     at a time, to the CTA that adds those tokens, parts in rank order (read from the
//     others' memory instead, 256 x 4096 x 4096 took 16.2 us for 11.8).
// Bound by: few tokens, the weights' bytes (64 tokens, 128256 x 4096, fp32 out: 52 us, 0.88 of HBM; one
// token, 14336 x 4096: 9.5-10.0 us, 0.46-0.48: start, first loads and end are half of it); many tokens,
// shared memory, which the copies fill with 35 KB a stage while the MMAs read both operands from
// it (8192 x 14336 x 4096: 145 us, 6.6 PFLOP/s, 0.88 of four times the bf16 rate; without
// the copies 132, with a quarter of the MMAs 120); short contractions, the outputs.
// Every wait is bounded as in the FP8 GEMM; what ran out is reported by rlq_check, and a CTA that gave up
// waits for its copies in flight before it leaves.  No pairs where RLQ_GEMM_PAIR=0.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "rlq_internal.h"
#include "rlq_tc.cuh"

namespace rlq {
namespace {

constexpr int BM = 128;          // rows of A of a CTA
constexpr int BK_BYTES = 128;    // bytes of a row's codes in a stage: 256 elements
constexpr int EPI_WARP0 = 2;
constexpr int EPI_GROUPS = 2;            // groups of four warps (a warp for each TMEM lane quarter)
constexpr int EPI_WARPS = 4 * EPI_GROUPS;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int STAGING_BYTES = EPI_WARPS * 4096;  // (pairs) 32 rows of 128 bytes a warp
constexpr int A_BYTES = BM * BK_BYTES;   // 16 KB
constexpr int AS_BYTES = 1024;           // a row tile's scales of a stage
constexpr int MAX_STAGES = 8;
constexpr int PREFETCH = 16;             // stages of weights that a CTA hints to L2 ahead
constexpr int NUM_BARS = 2 * MAX_STAGES + 7;
constexpr int BARS_BYTES = NUM_BARS * 8 + 16;
// tcgen05.mma kind::mxf4 instruction descriptor: A and B E2M1 (1 in bits 7-9 and 10-11), both
// K-major, N >> 3 in bits 17-22, E8M0 scales (bit 23), M >> 4 in bits 24-28; the scales of an
// instruction are bytes 0-1 or 2-3 of a row's word in tensor memory (bits 29-30 for A, 4-5
// for B: 0 or 2).
constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | (1u << 23);
constexpr uint32_t IDESC_HIGH = (2u << 29) | (2u << 4);

struct Params {
    void *y;
    int64_t ldy;
    int staged;                  // A is X, and y is stored by TMA; else A is W, and a lane stores its column of y
    int ragged;                  // (staged) y's rows end inside 16 bytes, the unit in which a TMA store is cut off
    int a_rows, b_rows;
    int kstages, last_steps;     // stages, and instructions (64 elements) of the last one
    int b_tiles, units, tile_b;  // tiles of B, (A tile, B tile) units, rows of a B tile
    int splits, kps;             // CTAs that share a unit, stages of each
    uint32_t splits_inv;         // 2^16 / splits, rounded up
    int stages, stage_bytes, b_bytes, bs_bytes, tx_bytes;
    int tmem_cols, buf1, sf_col, overlap;
    uint64_t timeout_ns;
    int withhold;                // (diagnostic) the first stage's loads are left out
};

template <bool kPair>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate)
{
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// A box on its way to L2 (a hint: no completion to wait for).
__device__ __forceinline__ void tma_prefetch_l2(const CUtensorMap *map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"((uint64_t)map), "r"(x), "r"(y)
                 : "memory");
}

// One lane of a warp whose lanes are together.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// mbar_wait by a whole warp, the same answer in every lane.  (The lanes stay together, so
// what the loops around it compute stays in uniform registers, which tcgen05 and TMA
// instructions take their operands from: issuing them from a thread of its own cost some
// 70 cycles each.)
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                               uint64_t limit_ns, uint32_t site)
{
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
        return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, limit_ns, site));
}

// A 512-byte scale tile (32 rows of 16 bytes) to four columns of tensor memory, the same in
// all four lane quarters (pair: in both CTAs, each from its own shared memory).
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr)
{
    // no swizzle; 8-row groups of 16-byte rows lie 128 bytes apart
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    if constexpr (kPair)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 16 bytes to a CTA of the cluster, counted by the barrier beside them.
__device__ __forceinline__ void st_async4(uint32_t addr, uint32_t bar, const uint32_t *v)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
                 : "memory");
}

// The cluster's barrier without an order of memory (a release would wait for this thread's
// part of a saturated memory system): what has to be seen behind it is either the
// initialisation of barriers, which has a fence of its own, or comes with a barrier's count.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <bool kF32>
__device__ __forceinline__ void store_out(const Params &p, int64_t at, float v)
{
    if constexpr (kF32)
        static_cast<float *>(p.y)[at] = v;
    else {
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
        static_cast<uint16_t *>(p.y)[at] = b;
    }
}

// A row's 128 bytes of outputs (32 fp32 or 64 bf16) to its place in a TMA box, 128-byte swizzle:
// 16-byte pieces, which eight neighbouring lanes spread over all banks.
template <bool kF32>
__device__ __forceinline__ void stage_row(uint32_t box, int lane, const uint32_t *lo, const uint32_t *hi)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (kF32) {
                w[j] = lo[4 * i + j];
            } else {
                const uint32_t *h = i < 4 ? lo + 8 * i : hi + 8 * (i - 4);
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(w[j])
                    : "f"(__uint_as_float(h[2 * j + 1])), "f"(__uint_as_float(h[2 * j])));
            }
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(box + (uint32_t)(lane * 128 + ((i ^ (lane & 7)) << 4))),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}

template <bool kPair, bool kF32>
__global__ void __launch_bounds__(THREADS)
    k_gemm_mxfp4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmAs, const __grid_constant__ CUtensorMap tmBs,
                 const __grid_constant__ CUtensorMap tmOut, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int STAGING = kPair ? STAGING_BYTES : 0;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + p.stages * p.stage_bytes + STAGING);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NUM_BARS);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t s0 = smem_u32(smem);
    auto stage = [&](int s) { return s0 + (uint32_t)(s * p.stage_bytes); };  // A codes, B codes, A scales, B scales
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[MAX_STAGES + s]); };
    auto tfull = [&](int b) { return smem_u32(&bars[2 * MAX_STAGES + b]); };
    auto tempty = [&](int b) { return smem_u32(&bars[2 * MAX_STAGES + 2 + b]); };
    const uint32_t shared_free = smem_u32(&bars[2 * MAX_STAGES + 4]), teardown = smem_u32(&bars[2 * MAX_STAGES + 5]);
    const uint32_t parts_bar = smem_u32(&bars[2 * MAX_STAGES + 6]);
    const uint32_t rank = kPair || p.splits > 1 ? cta_rank() : 0;
    const int group = kPair ? 2 : p.splits;  // CTAs that work on one unit
    const int unit0 = blockIdx.x / group, unit_step = gridDim.x / group;
    const int ks0 = kPair ? 0 : (int)rank * p.kps;
    const int ks1 = kPair ? p.kstages : min(ks0 + p.kps, p.kstages);
    auto a_row = [&](int u) { return (u / p.b_tiles) * (kPair ? 2 * BM : BM) + (kPair ? (int)rank * BM : 0); };
    auto b_row = [&](int u) { return (u % p.b_tiles) * p.tile_b; };
    // n / splits (exact below 2^16 / splits; four tokens of at most 256 are counted)
    auto over_splits = [&](int n) { return (int)((uint32_t)n * p.splits_inv >> 16); };
    auto columns = [&](int u) { return min(p.tile_b, p.b_rows - b_row(u)); };
    // the MMA's columns: whole steps of 16 (pair: 32, half of them each CTA's)
    auto mma_n = [&](int u) { return kPair ? (columns(u) + 31) & ~31 : (columns(u) + 15) & ~15; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), kPair ? 2 * EPI_WARPS : EPI_WARPS);
        }
        mbar_init(shared_free, kPair ? 8 : 4);  // the group that reads the shared columns
        mbar_init(teardown, 1);
        mbar_init(parts_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmAs);
        prefetch_tmap(&tmBs);
        if (!kPair && unit0 < p.units) {
            // The weights' first stages start their way to L2 before the kernels in front (as a
            // rule the tokens' quantizer) have finished: a hint, nothing is read until the wait below.
            const int ar = a_row(unit0), ahead = min(ks1, ks0 + PREFETCH);
            for (int ks = ks0; ks < ahead; ++ks) {
                tma_prefetch_l2(&tmA, ks * BK_BYTES, ar);
                tma_prefetch_l2(&tmAs, ks * 256, ar / BM);
            }
        }
    }
    pdl_begin();
    tc_fence_before();
    __syncthreads();
    if (group > 1)
        cluster_arrive_relaxed();  // this CTA's barriers are initialised
    if (kPair)
        cluster_wait();  // and the other's
    tc_fence_after();
    const uint32_t tmem = __reduce_or_sync(0xFFFFFFFFu, *tmem_slot);  // (in a uniform register)

    bool met = false;  // (a shared contraction) has seen every CTA's stages used up
    if (warp == 0) {
        // ------------------------------------------------ TMA producer ---
        const bool one = elect_one();
        int it = 0, s = 0;  // stages so far, and the next one's place in the ring
        uint32_t phase = 1;
        bool ok = true;
        for (int u = unit0; ok && u < p.units; u += unit_step) {
            const int ar = a_row(u), br = b_row(u);
            const int bc = br + (kPair ? (int)rank * (mma_n(u) / 2) : 0);  // this CTA's part of B
            for (int ks = ks0; ks < ks1; ++ks, ++it) {
                if (!mbar_wait_warp(empty(s), phase, abort_flag, p.timeout_ns, SITE_PRODUCER_EMPTY)) {
                    ok = false;
                    break;
                }
                if (one && !(p.withhold && it == 0)) {  // (withheld: nothing arrives on this stage's barrier)
                    const uint32_t a = stage(s), b = a + A_BYTES, as = b + (uint32_t)p.b_bytes, bs = as + AS_BYTES;
                    if constexpr (kPair) {
                        // both CTAs' copies complete on the even CTA's barrier
                        const uint32_t fb = cluster_addr(full(s), 0);
                        if (rank == 0)
                            mbar_arrive_expect_tx(full(s), 2u * (uint32_t)p.tx_bytes);
                        tma_load_2d_pair(a, &tmA, fb, ks * BK_BYTES, ar);
                        tma_load_2d_pair(b, &tmB, fb, ks * BK_BYTES, bc);
                        tma_load_2d_pair(as, &tmAs, fb, ks * 256, ar / BM);
                        tma_load_2d_pair(bs, &tmBs, fb, ks * 256, br / BM);
                    } else {
                        mbar_arrive_expect_tx(full(s), (uint32_t)p.tx_bytes);
                        tma_load_2d(a, &tmA, full(s), ks * BK_BYTES, ar);
                        tma_load_2d(b, &tmB, full(s), ks * BK_BYTES, br);
                        tma_load_2d(as, &tmAs, full(s), ks * 256, ar / BM);
                        tma_load_2d(bs, &tmBs, full(s), ks * 256, br / BM);
                    }
                }
                __syncwarp();
                if (++s == p.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        if (one) {
            // behind the MMA warp's last commit a normal run has consumed every copy; a
            // CTA that gave up waits (bounded) for those still in flight
            volatile uint32_t never = 0;
            mbar_wait(teardown, 0, &never, p.timeout_ns, SITE_TEARDOWN);
            if (!ok || *abort_flag || p.withhold) {
                int first = it > p.stages ? it - p.stages : 0;
                if (p.withhold && first == 0)
                    first = 1;
                // (pairs: both CTAs' copies complete on the even CTA's barriers, and neither CTA leaves
                // before the other)
                for (int j = first; (!kPair || rank == 0) && j < it; ++j)
                    mbar_wait(full(j % p.stages), (uint32_t)(j / p.stages) & 1u, &never, 20000000ull, SITE_DRAIN);
                if (kPair) {
                    // a stage that only one of the two asked for never completes: time to land
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 200000ull)
                        __nanosleep(1000);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------- MMA issuer ---
        if (!kPair || rank == 0) {
            const bool one = elect_one();
            int tc = 0, s = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = unit0; ok && u < p.units; u += unit_step, ++tc) {
                const int buf = tc & 1;
                // the buffer is read out (two tiles ago), and so are the columns that it shares with
                // the other one (the tile before)
                if (!mbar_wait_warp(tempty(buf), ((uint32_t)(tc >> 1) & 1u) ^ 1u, abort_flag, p.timeout_ns,
                                    SITE_MMA_TMEM_EMPTY) ||
                    (p.overlap && tc > 0 && !mbar_wait_warp(shared_free, (uint32_t)(tc - 1) & 1u, abort_flag,
                                                            p.timeout_ns, SITE_MMA_TMEM_EMPTY))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int n = mma_n(u);
                const uint32_t d = tmem + (uint32_t)(buf * p.buf1), sf = tmem + (uint32_t)p.sf_col;
                // (a tile of B that starts in the middle of a scale tile: 32 rows a column)
                const int skip = (b_row(u) & 127) >> 5;
                const uint32_t idesc = IDESC | ((uint32_t)(n >> 3) << 17) | ((uint32_t)((kPair ? 2 * BM : BM) >> 4) << 24);
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (!mbar_wait_warp(full(s), phase, abort_flag, p.timeout_ns, SITE_MMA_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (one) {
                        const uint32_t a = stage(s), b = a + A_BYTES, as = b + (uint32_t)p.b_bytes, bs = as + AS_BYTES;
                        const uint64_t ad = sw128_desc(a), bd = sw128_desc(b);
                        const int steps = ks + 1 == p.kstages ? p.last_steps : 4;
#pragma unroll
                        for (int t = 0; t < 2; ++t)  // 128 elements: columns 4 t of A's scales, 8 + 8 t of B's
                            if (2 * t < steps) {
                                copy_scales<kPair>(sf + 4 * t, as + 512 * t);
                                copy_scales<kPair>(sf + 8 + 8 * t, bs + 512 * t);
                                if (n + 32 * skip > 128)
                                    copy_scales<kPair>(sf + 12 + 8 * t, bs + 1024 + 512 * t);
                            }
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // 64 elements: 32 bytes along the rows
                            if (j < steps)
                                mma_mx<kPair>(d, ad + 2 * j, bd + 2 * j, idesc | (j & 1 ? IDESC_HIGH : 0u),
                                              sf + 4 * (j >> 1), sf + 8 + 8 * (j >> 1) + skip, ks > ks0 || j > 0 ? 1u : 0u);
                        tc_commit_t<kPair>(empty(s));
                        if (ks + 1 == ks1)
                            tc_commit_t<kPair>(tfull(buf));
                    }
                    __syncwarp();
                    if (++s == p.stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every MMA issued above has completed once this commit arrives
            if (one) {
                tc_commit_t<kPair>(teardown);
                volatile uint32_t never = 0;
                mbar_wait(teardown, 0, &never, 20000000ull, SITE_TEARDOWN);
            }
        }
        __syncwarp();
    } else {
        // --------------------------------------------------- epilogue ---
        // Pieces of 64 columns (single CTAs, which have no registers for them: 32), the two
        // groups of warps in turn.
        constexpr int PIECE = kPair ? 64 : 32, PIECES = 256 / PIECE;
        const int q = warp & 3;  // TMEM lane quarter of this warp
        const int g = (warp - EPI_WARP0) >> 2, row = q * 32 + lane;
        const uint32_t box = s0 + (uint32_t)(p.stages * p.stage_bytes + (warp - EPI_WARP0) * 4096);
        const uint64_t policy = l2_policy(false);
        int tc = 0;
        for (int u = unit0; u < p.units; u += unit_step, ++tc) {
            const int buf = tc & 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(tfull(buf), (uint32_t)(tc >> 1) & 1u, abort_flag, p.timeout_ns,
                                                   SITE_EPI_TMEM_FULL)))
                break;
            tc_fence_after();
            const int nc = columns(u);
            if (!kPair && p.splits > 1) {
                // every CTA's stages are used up: their memory takes the parts
                cluster_wait();
                cluster_arrive_relaxed();
                cluster_wait();
                met = true;
            }
            const int slots_max = over_splits((nc + 3) / 4 + p.splits - 1);
            const int64_t ar = a_row(u) + row, br = b_row(u);
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * p.buf1);
            // the columns that the other buffer has too come first: the first buffer's last piece, the second's first
            const int first = buf == 0 ? PIECES - 1 : 0;
            const bool shares = p.overlap && g == (first & 1);
            uint32_t r[PIECE / 32][32];
#pragma unroll 1
            for (int i = 0; i < PIECES / EPI_GROUPS; ++i) {
                const int c0 = PIECE * (shares ? (first + EPI_GROUPS * i) & (PIECES - 1) : g + EPI_GROUPS * i);
                if (c0 < nc) {
#pragma unroll
                    for (int h = 0; h < PIECE / 32; ++h)
                        tmem_ld32_async(taddr + (uint32_t)(c0 + 32 * h), r[h]);
#pragma unroll
                    for (int h = 0; h < PIECE / 32; ++h)
                        tmem_wait32(r[h]);
                }
                const bool last = i + 1 == PIECES / EPI_GROUPS;
                if (last || (i == 0 && shares)) {  // the accumulator, or what the other buffer has of it, is read out
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (i == 0 && shares) {
                            if constexpr (kPair)
                                mbar_arrive_cluster(cluster_addr(shared_free, 0));
                            else
                                mbar_arrive(shared_free);
                        }
                        if (last) {
                            if constexpr (kPair)
                                mbar_arrive_cluster(cluster_addr(tempty(buf), 0));
                            else
                                mbar_arrive(tempty(buf));
                        }
                    }
                }
                if (c0 >= nc)
                    continue;
                if (kPair && p.staged) {
#pragma unroll
                    for (int h = 0; h < (kF32 ? 2 : 1); ++h) {
                        const int x = (int)br + c0 + 32 * h, y = (int)ar - lane;
                        if (p.ragged && x + (kF32 ? 32 : 64) > p.b_rows) {
                            // the box that the end of y's rows cuts inside 16 bytes: element by element
                            if (ar < p.a_rows) {
                                const int64_t at = ar * p.ldy + x;
#pragma unroll
                                for (int j = 0; j < (kF32 ? 32 : 64); ++j)
                                    if (x + j < p.b_rows)
                                        store_out<kF32>(p, at + j, __uint_as_float(r[(kF32 ? h : j / 32) % (PIECE / 32)][j % 32]));
                            }
                            continue;
                        }
                        if (lane == 0)  // the copy engine has read the box
                            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        __syncwarp();
                        stage_row<kF32>(box, lane, r[h], r[PIECE / 32 - 1]);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0 && x < p.b_rows && y < p.a_rows) {
                            tma_store_2d_hint(&tmOut, box, x, y, policy);
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    }
                    continue;
                }
                // lane: a column of y, registers: its rows
#pragma unroll
                for (int h = 0; h < PIECE / 32; ++h) {
                    const int c = c0 + 32 * h, left = min(32, nc - c);
                    if (p.splits > 1) {
                        // this CTA's part, four tokens of a column at a time, to the CTA that adds
                        // those tokens: [part][four tokens][column]
                        const uint32_t at = s0 + (uint32_t)(((int)rank * slots_max * BM + row) * 16);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (4 * j < left) {
                                const int four = c / 4 + j, slot = over_splits(four);
                                const uint32_t to = (uint32_t)(four - slot * p.splits);
                                st_async4(cluster_addr(at + (uint32_t)(slot * (BM * 16)), to),
                                          cluster_addr(parts_bar, to), &r[h][4 * j]);
                            }
                    } else if (ar < p.a_rows) {
                        int64_t at = (br + c) * p.ldy + ar;
#pragma unroll
                        for (int j = 0; j < 32; ++j, at += p.ldy)
                            if (j < left)
                                store_out<kF32>(p, at, __uint_as_float(r[h][j]));
                    }
                }
            }
        }
        if (kPair && lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // stores complete before exit
        __syncwarp();
    }

    if (!kPair && p.splits > 1) {
        // One unit a cluster.  The warps that have met the others' barrier add the parts.
        if (!met) {
            cluster_wait();
            cluster_arrive_relaxed();
            cluster_wait();
        }
        if (warp >= EPI_WARP0) {
            const int nc = columns(unit0), fours = (nc + 3) / 4, slots_max = over_splits(fours + p.splits - 1);
            const int slots = over_splits(fours - (int)rank + p.splits - 1);  // of this CTA
            if (threadIdx.x == EPI_WARP0 * 32)
                mbar_arrive_expect_tx(parts_bar, (uint32_t)(slots * p.splits * BM * 16));
            bool ok = met && __all_sync(0xFFFFFFFFu, mbar_wait(parts_bar, 0, abort_flag, p.timeout_ns, SITE_EPI_TMEM_FULL));
            const int row = (warp & 3) * 32 + lane;
            const int64_t ar = a_row(unit0) + row;
            if (ok && ar < p.a_rows) {
                const int g = (warp - EPI_WARP0) >> 2;
                const float4 *part = reinterpret_cast<const float4 *>(smem) + g * BM + row;
                int m = 4 * ((int)rank + g * p.splits);
                int64_t at = (int64_t)(b_row(unit0) + m) * p.ldy + ar;
                for (int i = g; i < slots; i += EPI_GROUPS, part += EPI_GROUPS * BM, m += 4 * EPI_GROUPS * p.splits,
                         at += 4 * EPI_GROUPS * p.splits * p.ldy) {
                    float4 v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < p.splits)
                            v[c] = part[c * slots_max * BM];
                    float4 sum = v[0];
#pragma unroll
                    for (int c = 1; c < 8; ++c)
                        if (c < p.splits)
                            sum = make_float4(sum.x + v[c].x, sum.y + v[c].y, sum.z + v[c].z, sum.w + v[c].w);
                    store_out<kF32>(p, at, sum.x);
                    if (m + 1 < nc)
                        store_out<kF32>(p, at + p.ldy, sum.y);
                    if (m + 2 < nc)
                        store_out<kF32>(p, at + 2 * p.ldy, sum.z);
                    if (m + 3 < nc)
                        store_out<kF32>(p, at + 3 * p.ldy, sum.w);
                }
            }
            if (!ok) {  // parts may still be on their way here: give them time to land
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 200000ull)
                    __nanosleep(1000);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) {
        if (warp == 1) {
            if (rank == 1 && lane == 0) {
                // the even CTA's last commit: no MMA writes this CTA's tensor memory or reads its shared memory
                volatile uint32_t never = 0;
                mbar_wait(teardown, 0, &never, p.timeout_ns, SITE_TEARDOWN);
            }
            __syncwarp();
        }
    }
    if (group > 1) {  // no CTA leaves while another may still signal it
        cluster_arrive_relaxed();
        cluster_wait();
    }
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

// Zeros, where there is nothing to add.
template <bool kF32>
__global__ void __launch_bounds__(THREADS) k_zero_out(const Params p)
{
    pdl_begin();
    const int64_t M = p.b_rows, N = p.a_rows;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * THREADS)
        store_out<kF32>(p, i / N * p.ldy + i % N, 0.0f);
}

// ---------------------------------------------------------------- host ---

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Codes [rows][bytes], boxes of 128 bytes x box_rows, or (scales) tiles of 128 words, boxes of
// two tiles x box_rows row tiles; what lies outside arrives as zeros.
rlq_status encode(CUtensorMap *map, const uint8_t *base, bool scales, int64_t inner, int64_t rows, int64_t pitch, int box_rows)
{
    auto enc = encode_fn();
    if (!enc)
        return fail(RLQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {scales ? 256u : (cuuint32_t)BK_BYTES, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, scales ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                           const_cast<uint8_t *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           scales ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(RLQ_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d) for a [%lld x %lld] MXFP4 operand, pitch %lld",
                    (int)r, (long long)rows, (long long)inner, (long long)pitch);
    return RLQ_OK;
}

// Output [rows][cols] of y, boxes of 128 bytes x 32 rows, 128-byte swizzle.
rlq_status encode_out(CUtensorMap *map, void *y, bool f32, int64_t rows, int64_t cols, int64_t ld)
{
    auto enc = encode_fn();
    if (!enc)
        return fail(RLQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {f32 ? 32u : 64u, 32};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(RLQ_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d) for the [%lld x %lld] output", (int)r,
                    (long long)rows, (long long)cols);
    return RLQ_OK;
}

template <bool kPair, bool kF32>
rlq_status launch(const CUtensorMap *maps, const Params &p, int grid, int cluster, cudaStream_t st)
{
    const size_t smem = 1024 + (size_t)p.stages * p.stage_bytes + (kPair ? STAGING_BYTES : 0) + BARS_BYTES;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_status(e, "device query");
    static std::atomic<bool> set[64];
    if (!set[dev & 63].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(k_gemm_mxfp4<kPair, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e != cudaSuccess)
            return cuda_status(e, "cudaFuncSetAttribute(max dynamic shared memory)");
        // All of the SM's memory as shared memory, so that the next call's quantizer finds a CTA's room
        // beside this one whatever its ring takes (40 tokens, 2560 x 10240: 9.2 us; 11.2 with a split for 196 KB).
        e = cudaFuncSetAttribute(k_gemm_mxfp4<kPair, kF32>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return cuda_status(e, "cudaFuncSetAttribute(carve-out)");
        set[dev & 63].store(true, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, k_gemm_mxfp4<kPair, kF32>, maps[0], maps[1], maps[2], maps[3], maps[4], p),
                       "MXFP4 GEMM launch");
}

// Clusters of s single CTAs, one ([0][s]) or two ([1][s]) CTAs to an SM, that the current device runs at
// once: fewer than their CTAs would fit, since a cluster stays within a group of SMs (one GB300, alone on
// an SM: 76, 46, 36, 28, 23, 15 and 15 of 2 .. 8; others differ by one or two).
struct AtOnce {
    int n[2][9];
};

const AtOnce &clusters_at_once()
{
    static AtOnce known[64];
    static std::once_flag once[64];
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(once[dev & 63], [dev] {
        for (int two = 0; two < 2; ++two)
            for (int s = 1; s <= 8; ++s) {
                cudaLaunchAttribute attr;
                attr.id = cudaLaunchAttributeClusterDimension;
                attr.val.clusterDim.x = s;
                attr.val.clusterDim.y = 1;
                attr.val.clusterDim.z = 1;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)s);
                cfg.blockDim = dim3(THREADS);
                cfg.dynamicSmemBytes = two ? 232448 / 2 - 1024 : 232448;
                cfg.attrs = &attr;
                cfg.numAttrs = 1;
                // (asked of a kernel that takes no tensor memory: of the others the query allows one CTA to an SM)
                int n = 0;
                if (cudaFuncSetAttribute(k_zero_out<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448) !=
                        cudaSuccess ||
                    cudaOccupancyMaxActiveClusters(&n, k_zero_out<false>, &cfg) != cudaSuccess) {
                    cudaGetLastError();  // (not this call's: contractions are not shared)
                    n = 0;
                }
                known[dev & 63].n[two][s] = n;
            }
    });
    return known[dev & 63];
}

// Whether so many clusters run at once beside the kernels around them, which may keep some of the SMs: not
// the last tenth of the clusters, of five CTAs and more not the last sixth (16 tokens, 3584 x
// 18944 in 28 of 28 clusters of five 16.8 us, in fours 14.3; 100 tokens, 2560 x 10240 in 20 of
// 23 of six 12.8, in as many of two CTAs an SM 11.1).
bool at_once(const AtOnce &c, int64_t units, int s, bool two)
{
    const int64_t n = c.n[two][s];
    return s < 3 ? units <= n : s < 5 ? 10 * units <= 9 * n : 20 * units <= 17 * n;
}

// How a product is cut: CTA pairs with tiles of 256 rows of A x tile_b rows of B, or single CTAs with
// 128 output columns x tile_b tokens, a cluster of `splits` to a tile; `two` of them on an SM.
struct Plan {
    bool pair, two;
    int tile_b, splits;
};

// The cheapest by a model of a launch's microseconds, fitted to measurements: a start and an
// end that grow with the tile, per wave the stages one after the other (or, if that is longer, the
// operands and the outputs at the rates that they reach), and the joining of a shared contraction.
// Measured (us), the tokens' quantizer in front: 1 token, 14336 x 4096: 10.9 alone, 10.9 in twos, 14.5 in
// fours; 1, 5120 x 25600: 21.8 in twos, 17.8 in threes; 64, 2048 x 8192: 11.6 in twos, 9.3 in fours,
// 9.1 in fives; 100, 4096 x 4096: 10.1 in twos, 9.8 in fours.  The product alone: 256, 4096 x 4096: 8.7 in tiles of 64, 9.5 of 128, 11.3 of 256, 9.6 in
// pairs; 300, 1024 x 4096: 7.1 in tiles of 128 in fours, 8.9 in pairs; 1001, 5120 x 5120: 18.6 in
// pairs, 17.4 in pairs with tiles of 192, 21.4 alone; 1001, 3584 x 18944: 27.3, 24.8; 8192, 14336 x
// 4096: 147, 160; 8192, 8192 x 256: 22.6 in pairs, 43.8 alone (outputs not staged).
Plan make_plan(int64_t M, int64_t N, int64_t K, bool f32, int sms, bool pairs, bool staged)
{
    const int64_t kstages = (K + 255) / 256;
    const double operands = (double)(M + N) * (double)K * 17 / 32 / 6.2e6, out = (double)M * (double)N * (f32 ? 4 : 2);
    auto longer = [&](double waves, double per_wave, double out_rate) {
        const double moved = operands + out / out_rate;
        const double stages = waves * per_wave;
        // (where the bytes are the bound, the shorter chain of stages: 1, 4096 x 14336 by 8: 11.2, by 3: 12.1)
        return stages > moved ? stages : moved + 0.02 * stages;
    };
    const AtOnce &clusters = clusters_at_once();
    const double direct = f32 ? 4.5e6 : 2.9e6;  // bytes a microsecond of outputs stored by the lanes
    Plan best = {};
    double least = 1e300;
    // (a pair's ring is too short for few tokens: 1, 38912 x 1600: 9.4 alone, 14.1; without a device there
    // are no SMs, and the launch says so)
    for (int tile = 256; pairs && sms > 1 && M > 128 && tile >= 128; tile -= 64) {
        const int64_t rows = staged ? M : N, cols = staged ? N : M;
        const int64_t units = ((rows + 255) / 256) * ((cols + tile - 1) / tile), slots = sms / 2;
        const double cost = 4.4 + longer((double)((units + slots - 1) / slots),
                                         (double)kstages * (tile == 256 ? 0.35 : tile == 192 ? 0.30 : 0.28),
                                         !staged ? direct : tile == 256 ? 5.8e6 : 5.0e6);
        if (cost < least) {
            least = cost;
            best = {true, false, tile, 1};
        }
    }
    for (int tile = 64;; tile *= 2) {
        const int b = M < tile ? (int)M : tile;
        const int64_t units = (N + BM - 1) / BM * ((M + b - 1) / b);
        for (int s = 1; s <= 8; ++s) {
            // (every CTA has a part: the last one's begins before the stages end)
            const int64_t kps = (kstages + s - 1) / s;
            if (s > 1 && (kps < 2 || (s - 1) * kps >= kstages))
                continue;
            // (clusters, two CTAs on an SM: 1 token, 4608 x 8192 in fours: 8.9, in threes alone 9.6; but 2 tokens, 3584 x
            // 18944 in fives: 13.6, in fours alone 12.5, and 64, 2560 x 10240 in eights: 11.5, in fives alone 10.0)
            const bool two = s == 1 ? b <= 112 && (units > sms || kps <= 12) : b == 1 && !at_once(clusters, units, s, false);
            if (s > 1 && !at_once(clusters, units, s, two))
                continue;
            // (waves behind the first one share the memory system with others throughout: 1.35 of its time)
            const double waves = 1.35 * (double)((units * s + sms - 1) / sms) - 0.35;
            const double cost = 3.6 + 0.0075 * b + longer(waves, (double)kps * (0.26 + 0.0003 * b), direct) +
                                (s > 1 ? 0.6 + 0.008 * b : 0.0);
            if (cost < least) {
                least = cost;
                best = {false, two, b, s};
            }
        }
        if (M <= tile || tile == 256)
            break;
    }
    return best;
}

// The plan's tiles: (A tile, B tile) units for `slots` pairs, single CTAs or (two to an SM) twice as many.
struct Cut {
    Plan plan;
    bool staged;             // A is X, and y is stored by TMA; else A is W
    int64_t a_rows, b_rows;
    int tile_b;              // rows of a B tile
    int64_t a_tiles, b_tiles;
    int slots;
};

Cut make_cut(int64_t M, int64_t N, int64_t K, bool f32, bool pairs, bool aligned)
{
    const int sms = device_sms();
    Cut c;
    c.plan = make_plan(M, N, K, f32, sms, pairs, aligned);
    c.staged = c.plan.pair && aligned;
    c.a_rows = c.staged ? M : N;
    c.b_rows = c.staged ? N : M;
    c.tile_b = c.b_rows < c.plan.tile_b ? (int)c.b_rows : c.plan.tile_b;
    const int tile_a = c.plan.pair ? 2 * BM : BM;
    c.a_tiles = (c.a_rows + tile_a - 1) / tile_a;
    c.b_tiles = (c.b_rows + c.tile_b - 1) / c.tile_b;
    c.slots = c.plan.pair ? sms / 2 : c.plan.two ? 2 * sms : sms;
    return c;
}

}  // namespace

void gemm_mxfp4_cut(int64_t M, int64_t N, int64_t K, bool f32, bool aligned, int32_t *cut)
{
    const Cut c = make_cut(M, N, K, f32, pair_mode_enabled(), aligned);
    const int64_t units = c.a_tiles * c.b_tiles;
    cut[0] = c.plan.pair;
    cut[1] = c.staged;
    cut[2] = c.tile_b;
    cut[3] = c.plan.splits;
    cut[4] = c.plan.two;
    cut[5] = c.plan.splits > 1 ? 1 : (int32_t)((units + c.slots - 1) / c.slots);
}

rlq_status launch_gemm_mxfp4(const uint8_t *xq, int64_t ldxq, const uint8_t *xs, const uint8_t *wq, int64_t ldwq,
                             const uint8_t *ws, void *y, bool f32, int64_t ldy, int64_t M, int64_t N, int64_t K,
                             cudaStream_t st)
{
    Params p = {};
    p.y = y;
    p.ldy = ldy;
    if (K == 0) {
        const int sms = device_sms();
        p.a_rows = (int)N;
        p.b_rows = (int)M;
        const int64_t blocks = (M * N + THREADS - 1) / THREADS;
        return cuda_status(launch_pdl(f32 ? k_zero_out<true> : k_zero_out<false>,
                                      dim3((unsigned)(blocks < 6 * sms ? blocks : 6 * sms)), dim3(THREADS), 0, st, p),
                           "MXFP4 GEMM launch");
    }
    const int64_t ktiles = (K + 127) / 128;
    p.kstages = (int)((K + 255) / 256);
    p.last_steps = (int)((K - (int64_t)(p.kstages - 1) * 256 + 63) / 64);
    p.timeout_ns = wait_limit_ns();
    p.withhold = take_stall();
    const bool aligned = ((uintptr_t)y & 15) == 0 && ldy * (f32 ? 4 : 2) % 16 == 0;
    const Cut cut = make_cut(M, N, K, f32, pair_mode_enabled(), aligned);
    const Plan &plan = cut.plan;
    const bool pair = plan.pair;
    p.staged = cut.staged;
    p.ragged = N * (f32 ? 4 : 2) % 16 != 0;
    struct Operand {
        const uint8_t *q;
        int64_t ld;
        const uint8_t *s;
        int64_t rows;
    };
    const Operand x = {xq, ldxq, xs, M}, w = {wq, ldwq, ws, N};
    const Operand &A = p.staged ? x : w, &B = p.staged ? w : x;
    p.a_rows = (int)cut.a_rows;
    p.b_rows = (int)cut.b_rows;
    p.tile_b = cut.tile_b;
    p.b_tiles = (int)cut.b_tiles;
    if (cut.a_tiles * cut.b_tiles >= (int64_t)1 << 30)
        return fail(RLQ_ERR_UNSUPPORTED, "output of %lld x %lld has too many tiles", (long long)M, (long long)N);
    p.units = (int)(cut.a_tiles * cut.b_tiles);
    p.splits = plan.splits;
    p.kps = (p.kstages + p.splits - 1) / p.splits;

    const int n16 = pair ? (p.tile_b + 31) / 32 * 32 : (p.tile_b + 15) / 16 * 16;
    // scale tiles that a B tile reaches into (one of 192 rows may begin in the middle of one)
    const int box_b = pair ? n16 / 2 : p.tile_b, box_bs = p.tile_b > 128 ? 2 : 1;
    p.b_bytes = (pair ? n16 / 2 : n16) * BK_BYTES;
    p.bs_bytes = 1024 * box_bs;
    p.stage_bytes = (A_BYTES + p.b_bytes + AS_BYTES + p.bs_bytes + 1023) / 1024 * 1024;
    p.tx_bytes = A_BYTES + box_b * BK_BYTES + AS_BYTES + p.bs_bytes;
    // Tensor memory: two accumulators and 24 columns of scales.  Up to 112 columns fit in 256
    // of it and half of the shared memory, two CTAs to an SM: where there are more CTAs than
    // SMs (64 tokens, 128256 x 4096: 50.2 us, 51.5 with one an SM), and for short
    // contractions, whose next call then starts beside this one (1001 tokens, 1024 x 2048: 6.0
    // us back to back, 7.9 with one).  Long ones gain by the larger ring (64 tokens, 14336 x
    // 4096: 9.7 us, 10.3 with two).
    const bool two = plan.two;
    p.tmem_cols = two ? 256 : 512;
    p.sf_col = two ? 224 : 480;
    p.buf1 = n16 < 224 ? n16 : 224;
    p.overlap = n16 > 224;
    const int room = (two ? 232448 / 2 - 1024 : 232448) - 1024 - BARS_BYTES - (pair ? STAGING_BYTES : 0);
    p.stages = room / p.stage_bytes < MAX_STAGES ? room / p.stage_bytes : MAX_STAGES;
    p.splits_inv = (uint32_t)((65536 + p.splits - 1) / p.splits);
    CUtensorMap maps[5] = {};
    rlq_status r = encode(&maps[0], A.q, false, (K + 1) / 2, A.rows, A.ld, BM);
    if (r == RLQ_OK)
        r = encode(&maps[1], B.q, false, (K + 1) / 2, B.rows, B.ld, box_b);
    if (r == RLQ_OK)
        r = encode(&maps[2], A.s, true, ktiles * 128, (A.rows + 127) / 128, ktiles * 512, 1);
    if (r == RLQ_OK)
        r = encode(&maps[3], B.s, true, ktiles * 128, (B.rows + 127) / 128, ktiles * 512, box_bs);
    if (r == RLQ_OK && p.staged)
        r = encode_out(&maps[4], y, f32, M, N, ldy);
    if (r != RLQ_OK)
        return r;
    const int work = p.units < cut.slots ? p.units : cut.slots;
    if (pair)
        return f32 ? launch<true, true>(maps, p, 2 * work, 2, st) : launch<true, false>(maps, p, 2 * work, 2, st);
    const int grid = p.splits > 1 ? p.splits * p.units : work;
    return f32 ? launch<false, true>(maps, p, grid, p.splits, st) : launch<false, false>(maps, p, grid, p.splits, st);
}

cudaError_t take_mxfp4_error_word(cudaStream_t st, unsigned long long *word) { return take_error_word(st, word); }

}  // namespace rlq
