// The gated feed-forward block for few tokens (sm_103a): rlq_gemm_gated_fprop of a
// decode step, where the whole cost is one read of the two projections' codes.
//
//   g = X Wg^T, u = X Wu^T, a = g sigmoid(g) u, a (and g, u) to 1x128 FP8 codes
//
// A tile of the tcgen05 kernel is 128 rows of X, so with a few tokens it streams the
// weights through 128-column tiles on F / 128 SMs and leaves the rest idle.  Here a
// persistent cluster of four CTAs, two CTAs per SM, takes one 1x128 group of the output
// after another, 32 columns (32 gate and 32 up rows of W) a CTA, whose eight warps
// alternate over the 128-wide contraction blocks.  The products are mma.sync (16 x 8 x
// 16, fp16 in, fp32 out): E4M3 is exact in fp16, and since a contraction may be taken in
// any order, a thread's 16 consecutive bytes of a row serve as its operand elements of
// four products, for W and X alike, without any shuffle.  So each thread copies ahead
// (cp.async, its own slots of shared memory) what it will itself use, across the groups,
// and no barrier stands in the loop.  Tokens are the products' 8 columns.  Each block's
// sum is scaled in fp32, the warps' sums are added in order in shared memory, the group
// maxima are exchanged across the cluster while the next group's weights arrive.
//
// Bound by memory: 2 F K bytes of weight codes.  Measured back to back, one token: F =
// 14336, K = 4096 23.5 us (0.74 of the HBM rate; the tcgen05 kernel 24.6), 18944 x 3584
// 25 us (0.80; the same), 27648 x 5120 46.3 us (0.90; 54.2), 5120 x 5120 13.5 us (23.2);
// about 4 us of each are the first copies' and the last group's latency.  One CTA per SM with three times the ring: 25.9, 28.8,
// 48.0 (the GPU holds 36 such clusters, 112 groups take four rounds; with two CTAs per SM
// a round's stragglers have the SM's bandwidth to themselves).  16 tokens this way were
// no faster than the tcgen05 kernel, so more than 8 go there.
#include <cuda_runtime.h>

#include "rlq_elem.cuh"
#include "rlq_internal.h"

namespace rlq {
namespace {

constexpr int GRP = 128;
constexpr int COLS = 32;   // output columns per CTA
constexpr int WARPS = 8;
constexpr int TOKENS = 8;  // columns of a product, one per warp in the end
constexpr int CLUSTER = GRP / COLS;

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 16 E4M3 codes as 8 pairs of fp16 (exact).
__device__ __forceinline__ void to_f16(const uint4 &c, uint32_t (&h)[8])
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint16_t two = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"(two));
    }
}

// d += A (16 x 16) B (16 x 8), fp16 operands, fp32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float warp_max(float a)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    return a;
}

__device__ __forceinline__ float ld_cluster(const float *p, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct DecodeArgs {
    const uint8_t *xq;
    int64_t ldxq;
    const float *xs;
    int64_t ldxs;
    const uint8_t *wq;
    int64_t ldwq;
    const float *ws;
    int64_t ldws;
    uint8_t *aq;
    int64_t ldaq;
    float *as;
    int64_t ldas;
    uint8_t *guq;
    int64_t ldguq;
    float *gus;
    int64_t ldgus;
    int M;
    int64_t F;
    int kblocks;
};

// Shared-memory pitch of one output column's tokens (odd: conflict-free reads by column).
constexpr int PITCH = TOKENS + 1;
constexpr int DEPTH = 4;   // tiles in flight per warp
constexpr int RING_BYTES = DEPTH * 4 * 32 * WARPS * 16;
constexpr int SMEM = RING_BYTES + WARPS * 64 * PITCH * 4;
constexpr int CTAS_SM = 2;
static_assert(CTAS_SM * (SMEM + 2048) <= 228 * 1024, "shared memory of an SM");
static_assert(DEPTH % 4 == 0, "slot and tile index go together");
static_assert(TOKENS == WARPS, "a warp finishes one token");

// A warp's work is a sequence of 16-row tiles of 128-wide contraction blocks, four tiles
// a block, 64 bytes a thread each; DEPTH tiles are in flight.
__global__ void __launch_bounds__(32 * WARPS, CTAS_SM) k_gated_decode(const DecodeArgs p)
{
    extern __shared__ __align__(16) uint8_t smem[];  // the ring, then the warps' sums
    __shared__ float gmax[2][3][TOKENS];             // by parity of the group
    float *red = reinterpret_cast<float *>(smem + RING_BYTES);  // [warp][64 rows][PITCH]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int rank = blockIdx.x & (CLUSTER - 1), clusters = gridDim.x / CLUSTER;
    const int groups = (int)(p.F / GRP);
    const int64_t half = 8 * p.ldwq;
    // this thread's first byte of tile i (0, 1: gate rows, 2, 3: the up rows of the same columns)
    auto tile_row = [&](int group, int i) {
        return p.wq + ((i >> 1) * p.F + (int64_t)group * GRP + COLS * rank + 16 * (i & 1) + g) * p.ldwq + 16 * q;
    };
    int group = blockIdx.x / CLUSTER;
    // The weights' first lines start their way to L2 before the kernels in front have
    // finished (a hint: nothing is read until the wait).
    if (q == 0 && warp < p.kblocks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *r = tile_row(group, i) + (int64_t)warp * GRP;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(r));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(r + half));
        }
    pdl_begin();
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    constexpr uint32_t PIECE = 32 * WARPS * 16, SLOT = 4 * PIECE;
    const int nkb = p.kblocks > warp ? (p.kblocks - warp + WARPS - 1) / WARPS : 0;

    // The copies run ahead of the products through tiles, blocks and groups.
    int cg = nkb > 0 ? group : groups, cb = 0;
    const uint8_t *crow = tile_row(group, 0) + (int64_t)warp * GRP;  // of block cb of group cg
    const int64_t up = p.F * p.ldwq;
    // copies tile i of block cb of group cg
    auto copy_tile = [&](int i, int slot) {
        if (cg < groups) {
            const uint8_t *r = crow + (i >> 1) * up + (i & 1) * 2 * half;
            const uint32_t d = ring + slot * SLOT;
            copy16(d, r);
            copy16(d + PIECE, r + 64);
            copy16(d + 2 * PIECE, r + half);
            copy16(d + 3 * PIECE, r + half + 64);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (i == 3) {
            crow += WARPS * GRP;
            if (++cb == nkb) {
                cb = 0;
                cg += clusters;
                crow = tile_row(cg, 0) + (int64_t)warp * GRP;
            }
        }
    };
    auto load_x = [&](uint4 (&x)[2], float (&xs)[2], float (&ws)[2], int grp, int kb) {
        const int m = g, ms = 2 * q;
        const uint4 *r = reinterpret_cast<const uint4 *>(p.xq + (int64_t)m * p.ldxq + (int64_t)kb * GRP + 16 * q);
        x[0] = m < p.M ? __ldg(r) : make_uint4(0, 0, 0, 0);
        x[1] = m < p.M ? __ldg(r + 4) : make_uint4(0, 0, 0, 0);
        const float *rs = p.xs + (int64_t)kb * p.ldxs + ms;
        xs[0] = ms < p.M ? __ldg(rs) : 0.0f;
        xs[1] = ms + 1 < p.M ? __ldg(rs + 1) : 0.0f;
        ws[0] = __ldg(p.ws + (int64_t)grp * p.ldws + kb);
        ws[1] = __ldg(p.ws + (int64_t)(groups + grp) * p.ldws + kb);
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
        copy_tile(i & 3, i);
    uint4 x[2];
    float xs[2], ws[2];
    if (nkb > 0 && group < groups)
        load_x(x, xs, ws, group, warp);
    int slot0 = 0;  // slot of the block's first tile
    for (int par = 0; group < groups; group += clusters, par ^= 1) {
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = 0.0f;
        for (int b = 0; b < nkb; ++b) {
            uint4 cx[2];
            float cxs[2];
            const float cw[2] = {ws[0], ws[1]};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                cx[s] = x[s];
                cxs[s] = xs[s];
            }
            if (b + 1 < nkb)
                load_x(x, xs, ws, group, warp + WARPS * (b + 1));
            else if (group + clusters < groups)
                load_x(x, xs, ws, group + clusters, warp);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int slot = slot0 + i;
                asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
                uint4 w[2][2];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j >> 1][j & 1] =
                        *reinterpret_cast<const uint4 *>(smem + slot * SLOT + j * PIECE + threadIdx.x * 16);
                float part[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[j] = 0.0f;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    uint32_t lo[8], hi[8];
                    to_f16(w[0][s], lo);
                    to_f16(w[1][s], hi);
                    uint32_t xh[8];
                    to_f16(cx[s], xh);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma16816(part, lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1], xh[2 * j],
                                 xh[2 * j + 1]);
                }
                copy_tile(i, slot);  // (behind the uses of w: the slot's values are in registers)
                const float s0 = cxs[0] * cw[i >> 1], s1 = cxs[1] * cw[i >> 1];
                acc[i][0] = fmaf(part[0], s0, acc[i][0]);
                acc[i][1] = fmaf(part[1], s1, acc[i][1]);
                acc[i][2] = fmaf(part[2], s0, acc[i][2]);
                acc[i][3] = fmaf(part[3], s1, acc[i][3]);
            }
            slot0 = slot0 + 4 == DEPTH ? 0 : slot0 + 4;
        }
        // acc[i]: rows 16 i + g (+ 8), tokens 2 q (+ 1)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                red[(warp * 64 + 16 * i + g + 8 * (j >> 1)) * PITCH + 2 * q + (j & 1)] = acc[i][j];
        __syncthreads();
        // warp: a token; lane: an output column
        float gv = 0.0f, uv = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            gv += red[(w * 64 + lane) * PITCH + warp];
            uv += red[(w * 64 + 32 + lane) * PITCH + warp];
        }
        const float av = (gv * sigmoid2(make_float2(gv, gv)).x) * uv;
        const float ma = warp_max(fabsf(av));
        const float mg = p.guq ? warp_max(fabsf(gv)) : 0.0f, mu = p.guq ? warp_max(fabsf(uv)) : 0.0f;
        if (lane == 0) {
            gmax[par][0][warp] = ma;
            gmax[par][1][warp] = mg;
            gmax[par][2][warp] = mu;
        }
        __syncwarp();
        // Also: every warp has read the sums.  The maxima of this parity are written again
        // two groups on, behind the next group's barrier.
        cluster_barrier();
        const int64_t col = (int64_t)group * GRP + COLS * rank + lane;
        const int m = warp;
        if (m >= p.M)
            continue;  // (the same in all lanes; the next group's barrier is for all warps)
        // lane 4 k + r: matrix k's maximum in CTA r
        float v = lane < 12 ? ld_cluster(&gmax[par][lane >> 2][m], lane & 3) : 0.0f;
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
        const float s = group_scale(v), r = scale_rcp(s), pre = scale_pre(s);
        if (rank == 0) {
            if (lane == 0)
                p.as[(int64_t)group * p.ldas + m] = s;
            else if (p.guq && (lane == 4 || lane == 8))
                p.gus[((lane >> 3) * (int64_t)groups + group) * p.ldgus + m] = s;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k > 0 && !p.guq)
                break;
            const float rk = __shfl_sync(0xFFFFFFFFu, r, 4 * k), pk = __shfl_sync(0xFFFFFFFFu, pre, 4 * k);
            const float y = k == 0 ? av : k == 1 ? gv : uv;
            const uint8_t code = (uint8_t)e4m3x2((y * pk) * rk, 0.0f);
            if (k == 0)
                p.aq[(int64_t)m * p.ldaq + col] = code;
            else
                p.guq[(int64_t)m * p.ldguq + (k - 1) * p.F + col] = code;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    cluster_barrier();  // no CTA leaves while another may still read its maxima
}

}  // namespace

cudaError_t launch_gated_decode(const GemmArgs &a, cudaStream_t st)
{
    const DecodeArgs p = {a.A,  a.lda,  a.sa, a.ld_sa, a.B,   a.ldb,     a.sb,  a.sb_cstride, a.aq, a.ldaq,
                          a.as, a.ld_as, a.guq, a.ldguq, a.gus, a.ld_gus, (int)a.R, a.C, (int)(a.L / GRP)};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CLUSTER;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // clusters that are resident at once, looked up once per device
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    int n = resident[dev & 63].load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaFuncSetAttribute(k_gated_decode, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess)
            return e;
        cudaLaunchConfig_t query = cfg;
        query.gridDim = dim3((unsigned)(CTAS_SM * device_sms() / CLUSTER * CLUSTER));
        query.attrs = attr + 1;  // the cluster's shape alone
        query.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, k_gated_decode, &query);
        if (e != cudaSuccess)
            return e;
        if (n < 1)
            return cudaErrorLaunchOutOfResources;
        resident[dev & 63].store(n, std::memory_order_relaxed);
    }
    const int64_t groups = p.F / GRP;
    cfg.gridDim = dim3((unsigned)(CLUSTER * (groups < n ? groups : n)));
    return cudaLaunchKernelEx(&cfg, k_gated_decode, p);
}

}  // namespace rlq
