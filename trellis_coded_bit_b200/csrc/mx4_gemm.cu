// mx4_gemm.cu -- products of 4-bit microscaled matrices (mx4.cuh) on the
// fifth-generation tensor cores: exl3_mx4_matmul, exl3_mx4_linear,
// exl3_mx4_matmul_experts.
//
//     y[t, j] = sum_b 2^(ex[t, b] + ew[j, b]) sum_{l < 32} cx[t, 32b + l] cw[j, 32b + l]
//
// tcgen05.mma kind::mxf4.block_scale multiplies the codes and applies both
// scales itself (fp32 accumulators in TMEM), so nothing is decoded.  The
// weights are always the A operand (128 output channels in the TMEM lanes)
// and the tokens the B operand (N = TN columns, 16 .. 256), so that a single
// token costs a 16-column MMA instead of a 128-row one and one kernel serves
// both the decode (bound by the weights' bytes) and the prompt (bound by the
// tensor cores).
//
// Persistent and stream-K balanced: the work units are (128 channels x TN
// tokens, 256 columns of k) in tile order and CTA c of G owns units
// [cU/G, (c+1)U/G).  A tile whose units fall to several CTAs meets in the
// workspace: each segment writes its fp32 partial sums, the last to arrive
// (atomic ticket, no spinning) adds them in segment order and writes y, so
// results are deterministic.  A tile that is split is the last of exactly one
// CTA's range that begins it, so that CTA's number indexes its ticket.
//
// Warps: 0 TMA producer (weight and token codes, 128-byte swizzled boxes of
// 256 columns), 1 MMA issuer, 2..5 scales, 6..9 epilogue.  Scales are row-major
// in memory; the tensor core wants, per 128 columns and 128 rows, 512 bytes
// with row r's 4 scales at 16 (r % 32) + 4 (r / 32).  A scale thread owns a
// row: it copies 16 scales (512 columns) at a time into a private ring
// (cp.async, several steps ahead) and deals them out to the stages;
// tcgen05.cp then broadcasts a stage's scales to the TMEM columns that belong
// to the stage.
//
// All waits are bounded; a timeout is recorded in the workspace status word,
// and copies and MMAs in flight are drained before the CTA exits.
#include <cuda.h>

#include "dtypes.cuh"
#include "exl3_device.cuh"
#include "exl3_host.h"
#include "mx4.cuh"
#include "tcgen05.cuh"

namespace exl3 {

constexpr int kMxBM = 128;                       // output channels per tile (TMEM lanes)
constexpr int kMxBK = 256;                       // columns of k per unit: 128 bytes of codes
constexpr int kMxScaleWarp0 = 2, kMxEpiWarp0 = 6;
constexpr int kMxThreads = 32 * (kMxEpiWarp0 + 4);
constexpr int kMxABytes = kMxBM * kMxBK / 2;     // 16 KB
constexpr int kMxMaxExperts = 1024;
constexpr size_t kMxSyncArea = 64 * 1024;

// Sizes that follow from the token tile.
template <int TN>
struct MxTile {
    static constexpr int kBBytes = TN * kMxBK / 2;
    static constexpr int kBGroups = (TN + 127) / 128;          // 128-row groups of token scales
    static constexpr int kScaleBytes = 1024 + kBGroups * 1024;  // two 128-column chunks of 512 bytes per group
    static constexpr int kStageBytes = kMxABytes + kBBytes + kScaleBytes;
    static constexpr int kRowsPerThread = 1 + kBGroups;         // scale rows of a scale thread
    static constexpr int kDepth = TN > 128 ? 2 : 4;             // 512-column steps of scales in flight
    static constexpr int kRingBytes = kDepth * kRowsPerThread * 128 * 16;
    static constexpr int kStages = TN > 128 ? 4 : (TN > 64 ? 6 : (TN > 32 ? 7 : 8));
    static constexpr int kAcc = TN > 128 ? 1 : 2;               // accumulators in TMEM
    static constexpr int kScaleCols = 8 + 8 * kBGroups;         // TMEM columns of a stage's scales
    static constexpr int kAccCols = TN < 32 ? 32 : TN;
    static constexpr int kSmem = 1024 + 1024 + kStages * kStageBytes + kRingBytes;
    static_assert(kAcc * kAccCols + kStages * kScaleCols <= 512, "TMEM columns");
    static_assert(kSmem + 4 * (kMxMaxExperts + 1) <= 232448, "shared memory");
};

struct MxParams {
    const uint8_t *xs, *ws;     // scales, row-major
    const int32_t *offsets;     // [experts + 1] first token row of each expert, or null: one expert, all rows
    void *y;
    float *partials;            // [2 G][TN][128]
    uint32_t *counters;         // [G]
    uint32_t *status;
    int64_t rows;               // token rows
    int n, k, kb_count, experts, stride;
    uint64_t wait_ns;
};

struct MxBars {
    uint64_t tfull[8], sfull[8], empty[8];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem_slot;
    int epi_abort;
    int ticket;
};
static_assert(sizeof(MxBars) <= 1024, "barrier block");

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                         uint32_t sb, uint32_t accumulate)
{
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes) to 4 TMEM columns, repeated in the
// four lane quarters.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t saddr)
{
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3fffu) | (1ull << 16) | (8ull << 32) | (1ull << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// 16 bytes to shared memory, zeros if !valid (src is then not read).
__device__ __forceinline__ void cp_async16_zfill(void *dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(dst)), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

#define EXL3_TMEM_LD16(taddr, v)                                                                          \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14," \
                 "%15}, [%16];\n"                                                                          \
                 "tcgen05.wait::ld.sync.aligned;\n"                                                       \
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),     \
                   "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),              \
                   "=r"(v[13]), "=r"(v[14]), "=r"(v[15])                                                   \
                 : "r"(taddr)                                                                              \
                 : "memory")

// kind::mxf4: A and B e2m1, both K-major, e8m0 scales, M = 128, N = TN; the
// scale ids (which half of a 4-scale word) go in per MMA.
template <int TN>
__device__ __forceinline__ constexpr uint32_t mx_idesc(int half)
{
    return ((uint32_t)(2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(TN >> 3) << 17) | (1u << 23) |
           ((uint32_t)(kMxBM >> 4) << 24) | ((uint32_t)(2 * half) << 29);
}

// Where a tile lies: token rows [row, row_end), the weight row and the output
// channel of its first lane.
struct MxPlace {
    int64_t wrow;
    int64_t row, row_end;
    int ch;
};

// The rows of expert e, clamped into the buffer (the offsets are data).
__device__ __forceinline__ void mx_expert_rows(const MxParams &p, int e, int64_t &lo, int64_t &hi)
{
    lo = 0;
    hi = p.rows;
    if (p.offsets) {
        const int64_t a = p.offsets[e], b = p.offsets[e + 1];
        lo = a < 0 ? 0 : (a > p.rows ? p.rows : a);
        hi = b < lo ? lo : (b > p.rows ? p.rows : b);
    }
}

// Tile t: its expert from the tiles' prefix sums (smem), then token tiles
// fastest within a row of channels, so that neighbouring tiles share weights.
template <int TN>
__device__ __forceinline__ MxPlace mx_place(const MxParams &p, const uint32_t *first, uint32_t t)
{
    int lo = 0, hi = p.experts;  // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    MxPlace w;
    int64_t r0;
    mx_expert_rows(p, lo, r0, w.row_end);
    const uint32_t local = t - first[lo];
    const uint32_t tts = (uint32_t)((w.row_end - r0 + TN - 1) / TN);
    const uint32_t nt = local / tts;
    w.row = r0 + (int64_t)(local - nt * tts) * TN;
    w.ch = (int)nt * kMxBM;
    w.wrow = (int64_t)lo * p.n + w.ch;
    return w;
}

__device__ __forceinline__ uint32_t mx_begin(uint64_t c, uint64_t U, uint64_t G)
{
    return (uint32_t)(c * U / G);
}

// The CTA that owns unit u.
__device__ __forceinline__ uint32_t mx_owner(uint64_t u, uint64_t U, uint64_t G)
{
    return (uint32_t)(((u + 1) * G - 1) / U);
}

// Partial slot of CTA c's segment of the tile that begins at unit tb: its
// first segment uses 2c, its last 2c + 1.
__device__ __forceinline__ uint32_t mx_slot(uint32_t c, uint32_t tb, uint64_t U, uint64_t G)
{
    return mx_begin(c, U, G) >= tb ? 2 * c : 2 * c + 1;
}

__device__ __forceinline__ void mx_epi_sync()
{
    asm volatile("bar.sync 1, 128;\n" ::: "memory");
}

template <typename T, int TN>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_gemm_kernel(const MxParams p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap)
{
    using S = MxTile<TN>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    MxBars &bars = *reinterpret_cast<MxBars *>(smem);
    unsigned char *aring = smem + 1024;
    unsigned char *bring = aring + S::kStages * kMxABytes;
    unsigned char *scales = bring + S::kStages * S::kBBytes;
    unsigned char *sring = scales + S::kStages * S::kScaleBytes;
    uint32_t *first = reinterpret_cast<uint32_t *>(sring + S::kRingBytes);  // [experts + 1]
    volatile int *epi_abort = &bars.epi_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&bars.tfull[s], 1);
            mbar_init(&bars.sfull[s], 4);
            mbar_init(&bars.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.acc_full[b], 1);
            mbar_init(&bars.acc_empty[b], 4);
        }
        mbar_init(&bars.drain, 1);
        bars.epi_abort = 0;
        bars.ticket = 0;
        fence_mbar_init();
    }
    if (warp == 1)
        tmem_alloc(&bars.tmem_slot, 512);
    grid_dep_wait();
    if (warp == 0) {
        // prefix sums of the experts' tiles
        const uint32_t nts = (uint32_t)((p.n + kMxBM - 1) / kMxBM);
        uint32_t run = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            uint32_t v = 0;
            if (e0 + lane < p.experts) {
                int64_t lo, hi;
                mx_expert_rows(p, e0 + lane, lo, hi);
                v = (uint32_t)((hi - lo + TN - 1) / TN) * nts;
            }
            uint32_t incl = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
                incl += lane >= d ? o : 0;
            }
            if (e0 + lane < p.experts)
                first[e0 + lane] = run + incl - v;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0)
            first[p.experts] = run;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_slot;
    const uint32_t KB = (uint32_t)p.kb_count;
    const uint64_t U = (uint64_t)first[p.experts] * KB;
    // no more CTAs than units: with an empty range between two others a
    // tile's segments would be miscounted
    const uint64_t G = U < gridDim.x ? U : gridDim.x;
    const bool works = blockIdx.x < G;
    const uint32_t u0 = works ? mx_begin(blockIdx.x, U, G) : 0, u1 = works ? mx_begin(blockIdx.x + 1, U, G) : 0;
    const int nu = (int)(u1 - u0);

    if (warp == 0) {
        // ---------------------------------------------------- producer ---
        if (lane == 0 && nu > 0) {
            uint32_t t = u0 / KB;
            int kb = (int)(u0 - t * KB);
            MxPlace w = mx_place<TN>(p, first, t);
            int issued = 0;
            for (int i = 0; i < nu; ++i) {
                const int s = i % S::kStages;
                if (!mbar_wait(&bars.empty[s], ((uint32_t)(i / S::kStages) & 1u) ^ 1u, p.wait_ns)) {
                    record_timeout(p.status);
                    break;
                }
                mbar_arrive_expect_tx(&bars.tfull[s], kMxABytes + S::kBBytes);
                tma_load_2d(aring + s * kMxABytes, &wmap, kb * (kMxBK / 2), (int)w.wrow, &bars.tfull[s]);
                tma_load_2d(bring + s * S::kBBytes, &xmap, kb * (kMxBK / 2), (int)w.row, &bars.tfull[s]);
                issued = i + 1;
                if (++kb == (int)KB && i + 1 < nu) {
                    kb = 0;
                    w = mx_place<TN>(p, first, ++t);
                }
            }
            for (int i = (issued > S::kStages ? issued - S::kStages : 0); i < issued; ++i)
                if (!mbar_wait(&bars.tfull[i % S::kStages], (uint32_t)(i / S::kStages) & 1u, kDefaultWaitNs))
                    record_timeout(p.status);
        }
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer ---
        if (lane == 0 && nu > 0) {
            int kb = (int)(u0 % KB);
            int seg = 0;
            bool ok = true;
            for (int i = 0; i < nu; ++i) {
                const bool seg_start = i == 0 || kb == 0;
                const bool seg_end = i == nu - 1 || kb == (int)KB - 1;
                const int acc = seg % S::kAcc;
                if (seg_start && seg >= S::kAcc) {
                    if (!mbar_wait(&bars.acc_empty[acc], (uint32_t)(seg / S::kAcc - 1) & 1u, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                }
                const int s = i % S::kStages;
                const uint32_t par = (uint32_t)(i / S::kStages) & 1u;
                if (!mbar_wait(&bars.tfull[s], par, p.wait_ns) || !mbar_wait(&bars.sfull[s], par, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * S::kAccCols);
                const uint32_t tsa = tmem + (uint32_t)(S::kAcc * S::kAccCols + s * S::kScaleCols);
                const uint32_t tsb = tsa + 8;
                const uint32_t sc = smem_addr(scales + s * S::kScaleBytes);
                // chunk c's scales: weights at tsa + 4c, tokens at tsb + 4 groups c
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tmem_copy_scales(tsa + 4 * c, sc + 512 * c);
#pragma unroll
                    for (int g = 0; g < S::kBGroups; ++g)
                        tmem_copy_scales(tsb + 4 * (c * S::kBGroups + g), sc + 1024 + 512 * (c * S::kBGroups + g));
                }
                const uint32_t a0 = smem_addr(aring + s * kMxABytes);
                const uint32_t b0 = smem_addr(bring + s * S::kBBytes);
                const int left = p.k - kb * kMxBK;
                const int steps = left >= kMxBK ? 4 : (left + 63) / 64;  // 64 columns per MMA; none behind k
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < steps)
                        mma_mxf4(d, smem_desc(a0 + 32 * j, 16, 1024), smem_desc(b0 + 32 * j, 16, 1024),
                                 (j & 1) ? mx_idesc<TN>(1) : mx_idesc<TN>(0), tsa + 4 * (j >> 1),
                                 tsb + 4 * S::kBGroups * (j >> 1), (!seg_start || j) ? 1u : 0u);
                mma_commit(&bars.empty[s]);
                if (seg_end) {
                    mma_commit(&bars.acc_full[acc]);
                    ++seg;
                }
                if (++kb == (int)KB)
                    kb = 0;
            }
            if (!ok)
                record_timeout(p.status);
            // no MMA may still be writing TMEM when the CTA tears down
            mma_commit(&bars.drain);
            if (!mbar_wait(&bars.drain, 0, kDefaultWaitNs))
                record_timeout(p.status);
        }
    } else if (warp < kMxEpiWarp0) {
        // ------------------------------------------------------ scales ---
        // Thread r copies row r of the weights and rows r (and r + 128) of the
        // tokens, 512 columns per step; a segment's steps begin at the pair
        // that holds its first unit.
        const int r = threadIdx.x - 32 * kMxScaleWarp0;
        unsigned char *mine = sring + r * 16;  // [depth][row][128 threads][16 bytes]
        const uint32_t dst_off = (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
        const int kblocks = p.k / kMx4Block;
        // issue side: (tile, pair) of the next step to copy
        uint32_t ft = nu > 0 ? u0 / KB : 0;
        int fkb = nu > 0 ? (int)(u0 - ft * KB) : 0;
        MxPlace w;
        if (nu > 0)
            w = mx_place<TN>(p, first, ft);
        uint32_t fu = u0;
        auto fetch = [&](int slot) {
            if (fu < u1) {
                const int64_t col = (int64_t)(fkb >> 1) * 16;
                unsigned char *to = mine + slot * (S::kRowsPerThread * 2048);
                const bool aok = w.ch + r < p.n;
                cp_async16_zfill(to, aok ? p.ws + (w.wrow + r) * p.stride + col : p.ws, aok);
#pragma unroll
                for (int g = 0; g < S::kBGroups; ++g) {
                    const int64_t row = w.row + r + 128 * g;
                    const bool bok = r + 128 * g < TN && row < w.row_end;
                    cp_async16_zfill(to + (1 + g) * 2048, bok ? p.xs + row * p.stride + col : p.xs, bok);
                }
                // the units this step serves: to the end of the pair, the tile or the range
                uint32_t n2 = 2 - (uint32_t)(fkb & 1);
                if (fkb + (int)n2 > (int)KB)
                    n2 = KB - fkb;
                fu += n2;
                fkb += (int)n2;
                if (fkb == (int)KB && fu < u1) {
                    fkb = 0;
                    w = mx_place<TN>(p, first, ++ft);
                }
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };
        for (int d = 0; d < S::kDepth; ++d)
            fetch(d);
        int kb = nu > 0 ? (int)(u0 % KB) : 0;
        int slot = 0;
        uint4 cur[S::kRowsPerThread];
        for (int i = 0; i < nu; ++i) {
            if (i == 0 || (kb & 1) == 0) {
                // a new step: its copy is the oldest of kDepth in flight
                asm volatile("cp.async.wait_group %0;\n" ::"n"(S::kDepth - 1) : "memory");
#pragma unroll
                for (int q = 0; q < S::kRowsPerThread; ++q)
                    cur[q] = *reinterpret_cast<const uint4 *>(mine + (slot * S::kRowsPerThread + q) * 2048);
                fetch(slot);
                slot = slot + 1 == S::kDepth ? 0 : slot + 1;
            }
            const int s = i % S::kStages;
            if (!warp_wait_uniform(&bars.empty[s], ((uint32_t)(i / S::kStages) & 1u) ^ 1u, p.wait_ns)) {
                if (lane == 0)
                    record_timeout(p.status);
                break;
            }
            unsigned char *sc = scales + s * S::kScaleBytes + dst_off;
            const int left = kblocks - kb * (kMxBK / kMx4Block);  // scales that exist from this unit on
            const uint32_t m0 = left >= 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
            const uint32_t m1 = left >= 8 ? 0xffffffffu : (left <= 4 ? 0u : (1u << (8 * (left - 4))) - 1u);
#pragma unroll
            for (int q = 0; q < S::kRowsPerThread; ++q) {
                const uint32_t w0 = (kb & 1) ? cur[q].z : cur[q].x;
                const uint32_t w1 = (kb & 1) ? cur[q].w : cur[q].y;
                if (q == 0) {
                    *reinterpret_cast<uint32_t *>(sc) = w0 & m0;
                    *reinterpret_cast<uint32_t *>(sc + 512) = w1 & m1;
                } else {
                    *reinterpret_cast<uint32_t *>(sc + 1024 + 512 * (q - 1)) = w0 & m0;
                    *reinterpret_cast<uint32_t *>(sc + 1024 + 512 * (S::kBGroups + q - 1)) = w1 & m1;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars.sfull[s]);
            if (++kb == (int)KB)
                kb = 0;
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
    } else {
        // ---------------------------------------------------- epilogue ---
        const int quarter = warp & 3;  // TMEM lanes this warp may access
        const int r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        T *const y = reinterpret_cast<T *>(p.y);
        uint32_t u = u0;
        for (int seg = 0; u < u1; ++seg) {
            const uint32_t t = u / KB;
            const uint32_t tb = t * KB, te = tb + KB;
            const uint32_t se = te < u1 ? te : u1;
            const bool whole = u == tb && se == te;
            const MxPlace w = mx_place<TN>(p, first, t);
            const int acc = seg % S::kAcc;
            const bool ok = warp_wait(&bars.acc_full[acc], (uint32_t)(seg / S::kAcc) & 1u, p.wait_ns, 200);
            if (!ok && lane == 0) {
                record_timeout(p.status);
                *epi_abort = 1;
            }
            // the four warps agree, so that none is left at a barrier of the
            // others (only they write the flag, and only before this barrier)
            mx_epi_sync();
            const bool stop = *epi_abort != 0;
            mx_epi_sync();
            if (stop)
                break;
            tc_fence_after();
            const uint32_t d = tmem + lane_base + (uint32_t)(acc * S::kAccCols);
            const int64_t cols64 = w.row_end - w.row;
            const int cols = cols64 < TN ? (int)cols64 : TN;
            T *const yt = y + w.row * p.n + w.ch + r;
            const bool live = w.ch + r < p.n;
            bool finish = true;
            uint32_t c_lo = 0;
            int nseg = 1;
            if (!whole) {
                c_lo = mx_owner(tb, U, G);
                nseg = (int)(mx_owner(te - 1, U, G) - c_lo) + 1;
                float *slot = p.partials + (size_t)mx_slot(blockIdx.x, tb, U, G) * (TN * kMxBM) + r;
#pragma unroll 1
                for (int c = 0; c < cols; c += 16) {
                    uint32_t v[16];
                    EXL3_TMEM_LD16(d + c, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        __stcg(slot + (c + i) * kMxBM, __uint_as_float(v[i]));
                }
                __threadfence();
                mx_epi_sync();
                if (threadIdx.x == 32 * kMxEpiWarp0) {
                    const uint32_t prev = atomicAdd(&p.counters[c_lo], 1u);
                    const int last = prev == (uint32_t)(nseg - 1);
                    if (last) {
                        __threadfence();
                        p.counters[c_lo] = 0u;  // every segment has arrived: re-arm for the next call
                    }
                    bars.ticket = last;
                }
                mx_epi_sync();
                finish = bars.ticket != 0;
            }
            if (finish) {
#pragma unroll 1
                for (int c = 0; c < cols; c += 16) {
                    float v[16];
                    if (whole) {
                        uint32_t b[16];
                        EXL3_TMEM_LD16(d + c, b);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] = __uint_as_float(b[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] = 0.f;
                        for (int j = 0; j < nseg; ++j) {
                            const float *src =
                                p.partials + (size_t)mx_slot(c_lo + j, tb, U, G) * (TN * kMxBM) + c * kMxBM + r;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                v[i] += __ldcg(src + i * kMxBM);
                        }
                    }
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < cols)
                                yt[(int64_t)(c + i) * p.n] = from_f32<T>(v[i]);
                    }
                }
            }
            // hand the accumulator back to the MMA issuer
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars.acc_empty[acc]);
            u = se;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host ---

// The driver's tensor map encoder, looked up once (no link against libcuda).
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return (EncodeTiled)f;
    }();
    return fn;
}

// Map of a code matrix: rows of `bytes` bytes, boxes of 128 bytes x `box`
// rows, 128-byte swizzle, zeros outside.
static bool code_map(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t bytes, int box)
{
    const EncodeTiled fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box};
    const cuuint32_t steps[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)codes, dims, strides, boxes, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Token tile for `rows` tokens per expert: the narrowest that takes them in
// one tile, up to the widest.
static int mx_token_tile(int64_t rows)
{
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}

// Rows of an average expert, rounded up.
static int64_t mx_rows_each(int64_t rows, int64_t experts)
{
    return (rows + experts - 1) / experts;
}

static size_t mx_workspace(int64_t rows, int64_t experts)
{
    const int tn = mx_token_tile(mx_rows_each(rows, experts));
    return kMxSyncArea + (size_t)2 * num_sms() * tn * kMxBM * 4;
}

static bool valid_mx_sizes(int64_t m, int64_t k, int64_t n, int64_t experts)
{
    return valid_mx4_k(k) && valid_mx4_rows(m) && n >= 1 && n <= (int64_t)1 << 24 && experts >= 1 &&
           experts <= kMxMaxExperts && experts * n <= (int64_t)1 << 30;
}

template <typename T, int TN>
static exl3_status launch_mx(const MxParams &p, const CUtensorMap &wmap, const CUtensorMap &xmap, int ctas,
                             cudaStream_t s)
{
    auto kern = mx4_gemm_kernel<T, TN>;
    const int smem = MxTile<TN>::kSmem + 4 * (p.experts + 1);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             MxTile<TN>::kSmem + 4 * (kMxMaxExperts + 1)) != cudaSuccess)
        return EXL3_ERR_CUDA;
    if (launch_kernel(kern, dim3(ctas), dim3(kMxThreads), (size_t)smem, s, p, wmap, xmap) != cudaSuccess)
        return EXL3_ERR_CUDA;
    return launch_status();
}

template <typename T>
static exl3_status launch_mx_tile(int tn, const MxParams &p, const CUtensorMap &wmap, const CUtensorMap &xmap, int ctas,
                                  cudaStream_t s)
{
    switch (tn) {
    case 16: return launch_mx<T, 16>(p, wmap, xmap, ctas, s);
    case 32: return launch_mx<T, 32>(p, wmap, xmap, ctas, s);
    case 64: return launch_mx<T, 64>(p, wmap, xmap, ctas, s);
    case 128: return launch_mx<T, 128>(p, wmap, xmap, ctas, s);
    default: return launch_mx<T, 256>(p, wmap, xmap, ctas, s);
    }
}

static exl3_status check_mx(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, const void *y,
                            int dtype, int64_t m, int64_t k, int64_t n, int64_t experts)
{
    if (!valid_mx_sizes(m, k, n, experts) || (dtype != EXL3_F16 && dtype != EXL3_BF16))
        return EXL3_ERR_INVALID_ARG;
    if (m == 0)
        return EXL3_OK;
    if (!xc || !xs || !wc || !ws || !y || !aligned16(xc) || !aligned16(xs) || !aligned16(wc) || !aligned16(ws) ||
        !aligned16(y))
        return EXL3_ERR_INVALID_ARG;
    const size_t st = (size_t)mx4_scale_stride(k), yb = (size_t)m * (size_t)n * 2;
    const void *in[4] = {xc, xs, wc, ws};
    const size_t bytes[4] = {(size_t)m * (size_t)(k / 2), (size_t)m * st, (size_t)(experts * n) * (size_t)(k / 2),
                             (size_t)(experts * n) * st};
    for (int i = 0; i < 4; ++i)
        if (ranges_overlap(in[i], bytes[i], y, yb))
            return EXL3_ERR_INVALID_ARG;
    return EXL3_OK;
}

static exl3_status run_mx(const uint8_t *xc, const uint8_t *xs, const int32_t *offsets, const uint8_t *wc,
                          const uint8_t *ws, void *y, int dtype, int64_t m, int64_t k, int64_t n, int64_t experts,
                          void *workspace, cudaStream_t s)
{
    const int tn = mx_token_tile(mx_rows_each(m, experts));
    CUtensorMap wmap, xmap;
    if (!code_map(&wmap, wc, experts * n, k / 2, kMxBM) || !code_map(&xmap, xc, m, k / 2, tn))
        return EXL3_ERR_CUDA;
    MxParams p;
    p.xs = xs;
    p.ws = ws;
    p.offsets = offsets;
    p.y = y;
    p.partials = (float *)((unsigned char *)workspace + kMxSyncArea);
    p.counters = (uint32_t *)((unsigned char *)workspace + 256);
    p.status = (uint32_t *)workspace;
    p.rows = m;
    p.n = (int)n;
    p.k = (int)k;
    p.kb_count = (int)((k + kMxBK - 1) / kMxBK);
    p.experts = (int)experts;
    p.stride = (int)mx4_scale_stride(k);
    p.wait_ns = wait_limit_ns();
    // units fit 32 bits: at most (rows/TN + experts) tiles of each channel row
    const int64_t tiles = ((m + tn - 1) / tn + (experts > 1 ? experts : 0)) * ((n + kMxBM - 1) / kMxBM);
    if (tiles * p.kb_count >= (int64_t)1 << 31)
        return EXL3_ERR_UNSUPPORTED;
    const int64_t sms = num_sms();
    const int ctas = (int)(tiles * p.kb_count < sms ? tiles * p.kb_count : sms);
    return dtype == EXL3_F16 ? launch_mx_tile<__half>(tn, p, wmap, xmap, ctas, s)
                             : launch_mx_tile<__nv_bfloat16>(tn, p, wmap, xmap, ctas, s);
}

// Workspace of exl3_mx4_linear: the matmul's, then the quantised activations.
struct MxLinearPlan {
    size_t codes, scales, total;
};

static MxLinearPlan mx_linear_plan(int64_t m, int64_t k)
{
    MxLinearPlan pl;
    pl.codes = (mx_workspace(m, 1) + 255) / 256 * 256;
    pl.scales = pl.codes + ((size_t)m * (size_t)(k / 2) + 255) / 256 * 256;
    pl.total = pl.scales + (size_t)m * (size_t)mx4_scale_stride(k);
    return pl;
}

}  // namespace exl3

extern "C" size_t exl3_mx4_matmul_workspace_size(int64_t m, int64_t k, int64_t n)
{
    return exl3::valid_mx_sizes(m, k, n, 1) ? exl3::mx_workspace(m, 1) : 0;
}

extern "C" exl3_status exl3_mx4_matmul(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws,
                                       void *y, int dtype, int64_t m, int64_t k, int64_t n, void *workspace,
                                       size_t workspace_bytes, void *stream)
{
    using namespace exl3;
    const exl3_status st = check_mx(xc, xs, wc, ws, y, dtype, m, k, n, 1);
    if (st != EXL3_OK || m == 0)
        return st;
    if (!workspace || !aligned16(workspace) || workspace_bytes < mx_workspace(m, 1))
        return EXL3_ERR_WORKSPACE;
    return run_mx(xc, xs, nullptr, wc, ws, y, dtype, m, k, n, 1, workspace, (cudaStream_t)stream);
}

extern "C" size_t exl3_mx4_matmul_experts_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts)
{
    return exl3::valid_mx_sizes(rows, k, n, experts) ? exl3::mx_workspace(rows, experts) : 0;
}

extern "C" exl3_status exl3_mx4_matmul_experts(const uint8_t *xc, const uint8_t *xs, const int32_t *offsets,
                                               const uint8_t *wc, const uint8_t *ws, void *y, int dtype, int64_t rows,
                                               int64_t k, int64_t n, int64_t experts, void *workspace,
                                               size_t workspace_bytes, void *stream)
{
    using namespace exl3;
    const exl3_status st = check_mx(xc, xs, wc, ws, y, dtype, rows, k, n, experts);
    if (st != EXL3_OK || rows == 0)
        return st;
    if (!offsets || !aligned16(offsets) ||
        ranges_overlap(offsets, (size_t)(experts + 1) * 4, y, (size_t)rows * (size_t)n * 2))
        return EXL3_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < mx_workspace(rows, experts))
        return EXL3_ERR_WORKSPACE;
    return run_mx(xc, xs, offsets, wc, ws, y, dtype, rows, k, n, experts, workspace, (cudaStream_t)stream);
}

extern "C" size_t exl3_mx4_linear_workspace_size(int64_t m, int64_t k, int64_t n)
{
    return exl3::valid_mx_sizes(m, k, n, 1) ? exl3::mx_linear_plan(m, k).total : 0;
}

extern "C" exl3_status exl3_mx4_linear(const void *x, int dtype, const void *signs, int rotate, const uint8_t *wc,
                                       const uint8_t *ws, void *y, int64_t m, int64_t k, int64_t n, void *workspace,
                                       size_t workspace_bytes, void *stream)
{
    using namespace exl3;
    if (!valid_mx_sizes(m, k, n, 1) || (rotate && k % 128) || (dtype != EXL3_F16 && dtype != EXL3_BF16))
        return EXL3_ERR_INVALID_ARG;
    if (m == 0)
        return EXL3_OK;
    if (!x || !aligned16(x) || (signs && !aligned16(signs)) || !y ||
        ranges_overlap(x, (size_t)m * (size_t)k * 2, y, (size_t)m * (size_t)n * 2) ||
        (signs && ranges_overlap(signs, (size_t)k * 2, y, (size_t)m * (size_t)n * 2)))
        return EXL3_ERR_INVALID_ARG;
    const MxLinearPlan pl = mx_linear_plan(m, k);
    if (!workspace || !aligned16(workspace) || workspace_bytes < pl.total)
        return EXL3_ERR_WORKSPACE;
    uint8_t *base = (uint8_t *)workspace;
    uint8_t *xc = base + pl.codes, *xs = base + pl.scales;
    const exl3_status st = check_mx(xc, xs, wc, ws, y, dtype, m, k, n, 1);
    if (st != EXL3_OK)
        return st;
    const exl3_status q = exl3_mx4_quantize(x, dtype, signs, rotate, nullptr, 1, m, xc, xs, m, k, stream);
    if (q != EXL3_OK)
        return q;
    return run_mx(xc, xs, nullptr, wc, ws, y, dtype, m, k, n, 1, workspace, (cudaStream_t)stream);
}
