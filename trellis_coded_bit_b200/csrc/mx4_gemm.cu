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
// Persistent, one CTA per SM.  The work units are (128 channels x TN tokens, 512
// columns of k); above 128 tokens a tile is 256 channels x 256 tokens on a pair of
// CTAs (tcgen05 cta_group::2: each holds its 128 channels and half the tokens'
// codes, and the pair's MMAs read both), which moves a third fewer bytes per
// product.  mx_schedule says how tiles are shared out; where several workers share
// one, each writes its fp32 partial sums and the last to arrive (atomic ticket, no
// spinning) adds them in a fixed order, so results are deterministic.  Small
// products take tiles of fewer channels instead, each with all of k, and for a few
// tokens with parts of k side by side in one MMA (mx_split).
//
// Warps: 0 MMA issuer, 1 copies (TMA, 128-byte swizzled boxes of 256 columns), 2
// and 3 scales, 4 .. epilogue.  Scales are row-major in memory; the tensor core
// wants, per 128 columns and 128 rows, 512 bytes with row r's 4 scales at
// 16 (r % 32) + 4 (r / 32).  The scale warps load them a few units ahead, deal
// them out to the stages in that order, and tcgen05.cp broadcasts a stage's to the
// TMEM columns that belong to the stage.
//
// What bounds it: few tokens, the weights' bytes (32 x 8192 x 28672: 27 us, 4.6
// TB/s, of which 19 us are the bytes and most of the rest the first copy's 2.6 us,
// the start, and uneven SMs); many, the supply of the tensor cores at
// the ends of tiles (2048 x 8192 x 28672: 201 us, 4.8 PFLOP/s; within a tile a unit
// takes 1050 cycles, the MMAs' own time, and while the tile before is stored
// 2000).
//
// All waits are bounded; a timeout is recorded in the workspace status word,
// and copies, MMAs and arrivals in flight are drained before the CTA exits (of a
// pair: by both CTAs, see the end of the producer and of the kernel).
#include <cuda.h>
#include <math.h>

#include "dtypes.cuh"
#include "exl3_device.cuh"
#include "exl3_host.h"
#include "mx4.cuh"
#include "mx4_quantize.cuh"
#include "mx4_settle.h"
#include "tcgen05.cuh"

namespace exl3 {

constexpr int kMxBM = 128;                       // output channels per CTA's tile, at most (TMEM lanes)
constexpr int kMxBK = 512;                       // columns of k per unit: 16 scales of a row, two boxes of codes
constexpr int kMxBoxK = 256;                     // columns of a box: 128 bytes of codes, the swizzle's width
constexpr int kMxMmaWarp = 0, kMxTmaWarp = 1, kMxScaleWarp0 = 2, kMxEpiWarp0 = 4;
constexpr int kMxABytes = kMxBM * kMxBK / 2;     // 32 KB
constexpr int kMxMaxExperts = 512;
constexpr int kMxFuseRows = 2;                   // tokens that the product of a layer quantises itself
constexpr int kMxQuantWarps = 4;                 // warps that quantise them
constexpr int kMxFoldRows = 4;                   // tokens of a product whose tiles hold parts of k side by side
constexpr size_t kMxSyncArea = 64 * 1024;
// Shared memory of the experts' tables: each one's first tile and first row.
constexpr int mx_table_bytes(int experts)
{
    return 8 * (experts + 1);
}
constexpr int kMxSmemLimit = 232448 - mx_table_bytes(kMxMaxExperts);

// Sizes that follow from the token tile TN and the CTAs that share it (CG).
template <int TN, int CG>
struct MxTile {
    static constexpr int kBRows = TN / CG;                      // token rows in this CTA's shared memory
    static constexpr int kBBytes = kBRows * kMxBK / 2;
    static constexpr int kBGroups = (TN + 127) / 128;           // 128-row groups of token scales
    static constexpr int kScaleBytes = 2048 + kBGroups * 2048;  // four 128-column chunks of 512 bytes per group
    static constexpr int kStageBytes = kMxABytes + kBBytes + kScaleBytes;
    static constexpr int kScaleRows = TN > 128 ? 6 : 4;         // rows of scales of a scale warp's lane
    static constexpr int kDepth = 2;                            // units whose scales are loaded ahead
    static constexpr int kFit = (kMxSmemLimit - 2048) / kStageBytes;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kAcc = TN > 128 ? 1 : 2;               // accumulators in TMEM
    static constexpr int kScaleCols = 16 + 16 * kBGroups;       // TMEM columns of a stage's scales
    static constexpr int kAccCols = TN < 32 ? 32 : TN;
    static constexpr int kEpiWarps = TN >= 128 ? 8 : 4;         // each: 32 lanes x kEpiCols columns
    static constexpr int kEpiCols = TN / (kEpiWarps / 4);
    static constexpr int kWarps = kMxEpiWarp0 + kEpiWarps;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kFuseThreads = kThreads + 32 * (kMxQuantWarps - 1);  // one takes a scale warp's place
    static constexpr int kSmem = 2048 + kStages * kStageBytes;
    static_assert(kAcc * kAccCols + kStages * kScaleCols <= 512, "TMEM columns");
};

struct MxParams {
    const uint8_t *xs, *ws;     // scales, row-major
    const int32_t *offsets;     // [experts + 1] first token row of each expert, or null: one expert, all rows
    void *y;
    float *partials;            // [2 CTAs][TN / 4][128][4]
    uint32_t *counters;         // [split tiles, fewer than workers][CG]
    uint32_t *status;
    int64_t rows;               // token rows
    int n, k, experts, stride;
    int kb_count;               // units: of 512 columns of each part
    int bm;                     // output channels per CTA's tile: a multiple of 8; 128 with several experts or pairs
    int fold;                   // log2 of the parts of k side by side in a tile (FOLD, kMxFoldRows tokens at most; else 0)
    uint32_t most;              // workers that share a split tile, at most
    uint64_t wait_ns;
    // FUSE: the activations themselves
    const void *x;
    const __half *signs;
    int rotate;
};

struct MxBars {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem_slot;
    int epi_abort;
    int ticket;
    // CG = 2
    int failed;                  // a role of either CTA stopped early (set in both)
    uint32_t steps[kMxRoles];    // in the leader: steps that each role has done
};
static_assert(sizeof(MxBars) <= 1024, "barrier block");

// ------------------------------------------- instructions, by CTA group ---

#define EXL3_MX_MMA(cg)                                                                                          \
    asm volatile(                                                                                                \
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"                                                              \
        "tcgen05.mma.cta_group::" cg ".kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" \
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                          \
        : "memory")

template <int CG>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                         uint32_t sb, uint32_t accumulate)
{
    if constexpr (CG == 1)
        EXL3_MX_MMA("1");
    else
        EXL3_MX_MMA("2");
}

// 512 bytes of scales (32 rows of 16 bytes) to 4 TMEM columns, repeated in the
// four lane quarters (with CG = 2 in both CTAs, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t saddr)
{
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3fffu) | (1ull << 16) | (8ull << 32) | (1ull << 46);
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrives on `bar` (with CG = 2 on that of both CTAs) when the MMAs and copies
// issued so far are done.
template <int CG>
__device__ __forceinline__ void mx_commit(uint64_t *bar)
{
    if constexpr (CG == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void mx_tmem_alloc(uint32_t *slot)
{
    if constexpr (CG == 1) {
        tmem_alloc(slot, 512);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_addr(slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void mx_tmem_dealloc(uint32_t taddr)
{
    if constexpr (CG == 1)
        tmem_dealloc(taddr, 512);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(taddr) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;\n" ::: "memory");
}

// The barrier at `bar`'s place in the cluster's CTA 0.
__device__ __forceinline__ uint32_t leader_addr(uint64_t *bar)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(a) : "r"(smem_addr(bar)));
    return a;
}

// Arrives there.  What the arrival orders stays within this SM (its scales in
// shared memory and its accumulators in TMEM, which the pair's MMAs read and
// write on this SM), so the default scope is enough; a release at cluster scope
// waits for every load and store in flight and cost 1200 to 2000 cycles a unit.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(leader_addr(bar)) : "memory");
}

// Stores a word at the place of `at` in the cluster's CTA `rank`; visible there
// after the next cluster_sync.
__device__ __forceinline__ void store_in_cta(void *at, uint32_t rank, uint32_t v)
{
    asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, %1;\nst.shared::cluster.u32 [a], %2;\n}\n" ::"r"(
                     smem_addr(at)),
                 "r"(rank), "r"(v)
                 : "memory");
}

// A role of the pair (mx4_settle.h) has ended after `steps` steps.
__device__ __forceinline__ void mx_role_done(MxBars &bars, int role, uint32_t steps)
{
    if ((threadIdx.x & 31) == 0)
        store_in_cta(&bars.steps[role], 0, steps);
}

// A role stopped before its time: the timeout is recorded, and both CTAs of a
// pair learn of it.
template <int CG>
__device__ __forceinline__ void mx_failed(MxBars &bars, uint32_t *status)
{
    record_timeout(status);
    if constexpr (CG == 2) {
        store_in_cta(&bars.failed, 0, 1u);
        store_in_cta(&bars.failed, 1, 1u);
    }
}

// The leader's producer warp, when all roles of the pair have ended and one of
// them early: completes the stages' barriers in place of the roles that stopped
// and waits until every copy that either CTA began has landed.
__device__ __forceinline__ void mx_settle_pair(MxBars &bars, uint32_t stages, uint32_t bytes)
{
    uint32_t first, end;
    mx_debt_range(bars.steps, stages, first, end);
    for (uint32_t i = first; i < end; ++i) {
        uint64_t *const bar = &bars.full[i % stages];
        const MxDebt d = mx_debt(bars.steps, i, bytes);
        if ((threadIdx.x & 31) == 0) {
            if (d.tx > 0)
                asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(smem_addr(bar)), "r"(d.tx) : "memory");
            if (d.tx < 0)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(smem_addr(bar)), "r"(-d.tx) : "memory");
            for (uint32_t j = 0; j < d.arrivals; ++j)
                mbar_arrive(bar);
        }
        __syncwarp();
        if (!warp_wait_uniform(bar, (i / stages) & 1u, kDefaultWaitNs))
            break;  // (the limit is long enough for all that is in flight)
    }
}

// True in one lane of the converged warp.  The MMA issuer runs its loop with
// the whole warp and elects the lane only around the instructions: inside an
// `if (lane == 0)` the compiler cannot see that the operands are uniform, and
// a unit's issue took 950 cycles instead of the tensor core's 520.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// A box of codes into this CTA's shared memory; its bytes count on `bar`, with
// CG = 2 the leader's (a shared::cluster address).
template <int CG>
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                smem_addr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
            "%3}], [%4];\n" ::"r"(smem_addr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
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

// kind::mxf4: A and B e2m1, both K-major, e8m0 scales, M = 128 per CTA, N = TN;
// `half` selects the scales within a word of four.
template <int TN, int CG>
__device__ __forceinline__ constexpr uint32_t mx_idesc(int half)
{
    return ((uint32_t)(2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(TN >> 3) << 17) | (1u << 23) |
           ((uint32_t)((kMxBM * CG) >> 4) << 24) | ((uint32_t)(2 * half) << 29);
}

// Where a tile lies: token rows [row, row_end), the weight row and the output
// channel of the first lane (of CTA 0 where two share the tile).
struct MxPlace {
    int64_t wrow;
    int64_t row, row_end;
    int ch;
};

// The experts' tables in shared memory: the first tile and the first row of
// each, both with one more entry.
struct MxTables {
    const uint32_t *tile, *row;
    int experts;
};

// An offset clamped into the buffer (the offsets are data).
__device__ __forceinline__ uint32_t mx_row(const MxParams &p, int e)
{
    const int64_t r = p.offsets[e];
    return (uint32_t)(r < 0 ? 0 : (r > p.rows ? p.rows : r));
}

// Tile t: its expert by bisection, then token tiles fastest within a row of
// channels, so that neighbouring tiles share weights.
template <int TN, int CG>
__device__ __forceinline__ MxPlace mx_place(const MxParams &p, const MxTables &tab, uint32_t t)
{
    int lo = 0, hi = tab.experts;  // tile[lo] <= t < tile[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.tile[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const uint32_t r0 = tab.row[lo], r1 = tab.row[lo + 1];
    const uint32_t local = t - tab.tile[lo];
    const uint32_t tts = (r1 - r0 + TN - 1) / TN;
    const uint32_t nt = local / tts;
    MxPlace w;
    w.row = (int64_t)r0 + (int64_t)(local - nt * tts) * TN;
    w.row_end = r1;
    w.ch = (int)nt * (p.bm * CG);
    w.wrow = (int64_t)lo * p.n + w.ch;
    return w;
}

// ------------------------------------------------------------ schedule ---
//
// T tiles on G workers (a CTA, or the pair of CTAs that shares a tile).  The
// last T mod G tiles are split over the workers along k and done first, so that
// the sums meet while the whole tiles run.  Then worker c takes the whole tiles
// c, c + G, ...: at any time the workers are on neighbouring tiles, which share
// weights, so that these come from memory once.  (With contiguous shares of the
// tiles instead, 74 pairs held 74 different rows of weights: 2048 x 8192 x 18944
// took 241 us, waiting 3.4 us for each copy.)
//
// A split tile has at most `most` workers: its last one reads a partial sum from
// each (mx_most_workers, on the host).
//
// Split tiles: `even` gives each tile floor or ceil(W / tiles) workers of its
// own, so a worker has one segment and waits for one sum; otherwise the units
// (tile, 512 columns) in order are cut into equal shares, and a worker may end
// one tile and begin the next.  Even is taken where its longest segment is at
// most one unit longer (4096 channels, k = 4096: 2 units either way).
struct MxSched {
    uint32_t worker, G, KB;
    uint32_t whole;      // whole tiles of each worker
    uint32_t split0;     // first split tile
    uint32_t splits;     // split tiles
    uint32_t U, W;       // their units, the workers that share them
    uint32_t u0, u1;     // this worker's units
    bool even;
    int split_segs, segs;
};

// Part [k0, k1) of tile t.
struct MxSeg {
    uint32_t t;
    int k0, k1;
};

// (32 bits are enough: there are fewer split tiles than workers, so the
// products stay below workers^2 2^22/256.)
__device__ __forceinline__ uint32_t mx_begin(const MxSched &m, uint32_t c)
{
    return c * m.U / m.W;
}

// even: the first worker of split tile i.
__device__ __forceinline__ uint32_t mx_first_worker(const MxSched &m, uint32_t i)
{
    return i * m.W / m.splits;
}

// The workers of split tile i: [lo, lo + n).
__device__ __forceinline__ void mx_workers(const MxSched &m, uint32_t i, uint32_t &lo, int &n)
{
    if (m.even) {
        lo = mx_first_worker(m, i);
        n = (int)(mx_first_worker(m, i + 1) - lo);
    } else {
        const uint32_t b = i * m.KB;
        lo = ((b + 1) * m.W - 1) / m.U;
        n = (int)(((b + m.KB) * m.W - 1) / m.U - lo) + 1;
    }
}

// Partial slot of worker c's segment of split tile i: its first segment uses
// 2c, its second 2c + 1.
__device__ __forceinline__ uint32_t mx_slot(const MxSched &m, uint32_t c, uint32_t i)
{
    return m.even || mx_begin(m, c) >= i * m.KB ? 2 * c : 2 * c + 1;
}

__device__ __forceinline__ MxSched mx_schedule(uint32_t tiles, uint32_t KB, uint32_t workers, uint32_t worker, uint32_t most)
{
    MxSched m;
    m.worker = worker;
    m.G = workers;
    m.KB = KB;
    m.whole = tiles / workers;
    m.split0 = m.whole * workers;
    m.splits = tiles - m.split0;
    m.U = m.splits * KB;
    // no more workers than units (with an empty share between two others a
    // tile's segments would be miscounted), and `most` for a tile
    m.W = m.U < workers ? m.U : workers;
    m.W = m.W < m.splits * most ? m.W : m.splits * most;
    m.u0 = m.u1 = 0;
    m.split_segs = 0;
    m.even = false;
    if (worker < m.W) {
        const uint32_t least = m.W / m.splits;  // workers of a tile, at least
        m.even = (KB + least - 1) / least <= (m.U + m.W - 1) / m.W + 1;
        if (m.even) {
            const uint32_t i = ((worker + 1) * m.splits - 1) / m.W;
            uint32_t lo;
            int n;
            mx_workers(m, i, lo, n);
            m.u0 = i * KB + (worker - lo) * KB / (uint32_t)n;
            m.u1 = i * KB + (worker - lo + 1) * KB / (uint32_t)n;
        } else {
            m.u0 = mx_begin(m, worker);
            m.u1 = mx_begin(m, worker + 1);
        }
        m.split_segs = (int)((m.u1 - 1) / KB - m.u0 / KB) + 1;
    }
    m.segs = m.split_segs + (int)m.whole;
    return m;
}

__device__ __forceinline__ MxSeg mx_seg(const MxSched &m, int i)
{
    MxSeg g;
    if (i >= m.split_segs) {
        g.t = m.worker + (uint32_t)(i - m.split_segs) * m.G;
        g.k0 = 0;
        g.k1 = (int)m.KB;
    } else {
        const uint32_t tile = m.u0 / m.KB + (uint32_t)i, b = tile * m.KB;
        g.t = m.split0 + tile;
        g.k0 = b < m.u0 ? (int)(m.u0 - b) : 0;
        g.k1 = b + m.KB < m.u1 ? (int)m.KB : (int)(m.u1 - b);
    }
    return g;
}

// ------------------------------------------------------------ epilogue ---

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    T v[2] = {from_f32<T>(a), from_f32<T>(b)};
    uint32_t r;
    memcpy(&r, v, 4);
    return r;
}

// Stores 8 tokens x 32 channels: v[i] holds the lane's channel of tokens 2i and
// 2i + 1.  Three butterfly exchanges (lanes 1, 2, 4 apart) turn 8 tokens of one
// channel into 8 channels of one token, so that 4 lanes store the 64 contiguous
// bytes of a token's 32 channels (`wide`: y's rows are 16-byte aligned).
// Otherwise each lane stores its own channel 8 times.  yt: y at the first token
// and the warp's first channel; ch_left: channels of y from there on.
// FULL: 8 tokens and 32 channels exist and rows are aligned; without branches
// the exchanges of several calls overlap.
template <typename T, bool FULL = false>
__device__ __forceinline__ void mx_store8(T *yt, int64_t n, const uint32_t *v, int tokens, int ch_left, bool wide)
{
    const int lane = threadIdx.x & 31;
    if (FULL || wide) {
        // lanes 1 apart: register i becomes (channel pair, token 2i + (lane & 1))
        const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
        uint32_t a[4], c[4], e[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            // the halves the neighbour needs, of two registers at once
            const uint32_t give = __byte_perm(v[i], v[i + 1], b0 ? 0x5410 : 0x7632);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
            a[i] = b0 ? __byte_perm(got, v[i], 0x7610) : __byte_perm(v[i], got, 0x5410);
            a[i + 1] = b0 ? __byte_perm(got, v[i + 1], 0x7632) : __byte_perm(v[i + 1], got, 0x7610);
        }
        // lanes 2 apart: register pairs (0, 1) and (2, 3); afterwards c[2h], c[2h + 1]
        // are 4 channels of token 4h + 2 (b1) + b0
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? a[2 * h] : a[2 * h + 1], 2);
            c[2 * h] = b1 ? got : a[2 * h];
            c[2 * h + 1] = b1 ? a[2 * h + 1] : got;
        }
        // lanes 4 apart: 8 channels of token 4 (b2) + 2 (b1) + b0
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b2 ? c[h] : c[2 + h], 4);
            e[h] = b2 ? got : c[h];
            e[2 + h] = b2 ? c[2 + h] : got;
        }
        const int token = lane & 7, group = lane & 24;
        if (FULL || (token < tokens && group < ch_left))
            *reinterpret_cast<uint4 *>(yt + token * n + group) = make_uint4(e[0], e[1], e[2], e[3]);
    } else if (lane < ch_left) {
        uint16_t *q = reinterpret_cast<uint16_t *>(yt + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < tokens)
                q[i * n] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
}

template <int TN, int CG>
__device__ __forceinline__ void mx_epi_sync()
{
    asm volatile("bar.sync 1, %0;\n" ::"n"(32 * MxTile<TN, CG>::kEpiWarps) : "memory");
}

// Hands accumulator `acc` back to the MMA issuer, one arrival a warp.
template <int CG>
__device__ __forceinline__ void mx_release(MxBars &bars, int acc)
{
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        if constexpr (CG == 1)
            mbar_arrive(&bars.acc_empty[acc]);
        else
            mbar_arrive_leader(&bars.acc_empty[acc]);
    }
}

// Segment `seg` of this worker.  Returns false if its accumulators never came
// (the caller stops).
template <typename T, int TN, int CG, bool FOLD>
__device__ __forceinline__ bool mx_epilogue(const MxParams &p, MxBars &bars, const MxTables &tab, const MxSched &sched,
                                            uint32_t tmem, int seg, uint32_t rank)
{
    using S = MxTile<TN, CG>;
    constexpr int kCols = S::kEpiCols;
    volatile int *epi_abort = &bars.epi_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3;                                  // TMEM lanes this warp may access
    const int c0 = (warp - kMxEpiWarp0) / 4 * kCols;              // its columns
    const MxSeg g = mx_seg(sched, seg);
    const bool whole = g.k0 == 0 && g.k1 == (int)sched.KB;
    const MxPlace w = mx_place<TN, CG>(p, tab, g.t);
    const int acc = seg % S::kAcc;
    const uint32_t par = (uint32_t)(seg / S::kAcc) & 1u;
    bool ok = true;
    if (lane == 0) {
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(&bars.acc_full[acc], par)) {
            if (global_ns() - t0 > p.wait_ns) {
                ok = false;
                break;
            }
        }
        if (!ok) {
            mx_failed<CG>(bars, p.status);
            *epi_abort = 1;
        }
    }
    // the epilogue warps agree, so that none is left at a barrier of the
    // others (only they write the flag, and only before this barrier)
    __syncwarp();
    mx_epi_sync<TN, CG>();
    const bool stop = *epi_abort != 0;
    mx_epi_sync<TN, CG>();
    if (stop)
        return false;
    mbar_wait(&bars.acc_full[acc], par, kDefaultWaitNs);  // complete: every lane observes it
    tc_fence_after();

    const uint32_t d = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * S::kAccCols + c0);
    const int64_t cols64 = w.row_end - w.row - c0;
    const int cols = cols64 < kCols ? (int)cols64 : kCols;         // this warp's tokens (may be <= 0)
    const int ch = w.ch + (int)rank * kMxBM + quarter * 32;        // the warp's first channel
    const int ch_end = w.ch + ((int)rank + 1) * p.bm;             // of this CTA's tile
    const int ch_left = (ch_end < p.n ? ch_end : p.n) - ch;        // may be <= 0
    const bool wide = (p.n & 7) == 0;
    T *const y = reinterpret_cast<T *>(p.y) + (w.row + c0) * p.n + ch;

    if constexpr (FOLD) {
        // Each part's sums lie in its own lanes and columns; they meet in
        // shared memory, added in the order of k.  (The tile is whole, and the
        // barriers above keep the sums of the tile before until they are read.)
        __shared__ float sums[4][kMxFoldRows][32];
        const int warps = 4 >> p.fold;                // warps of a part
        const int part = quarter >> (2 - p.fold);
        uint32_t b[16];
        EXL3_TMEM_LD16(d + part * (16 >> p.fold), b);  // (behind the tokens' columns: not used)
        mx_release<CG>(bars, acc);
#pragma unroll
        for (int i = 0; i < kMxFoldRows; ++i)
            sums[quarter][i][lane] = __uint_as_float(b[i]);
        mx_epi_sync<TN, CG>();
        if (part == 0 && lane < ch_left) {
#pragma unroll
            for (int i = 0; i < kMxFoldRows; ++i) {
                if (i < cols) {
                    float s = sums[quarter][i][lane];
                    for (int j = 1; j < 1 << p.fold; ++j)
                        s += sums[quarter + j * warps][i][lane];
                    y[(int64_t)i * p.n + lane] = from_f32<T>(s);
                }
            }
        }
        return true;
    }

    if constexpr (sizeof(T) == 4) {
        // fp32: a warp's 32 channels of a token are 128 contiguous bytes as
        // they come from TMEM
        if (whole) {
            constexpr int kLoad = kCols % 32 == 0 ? 32 : 16, kStep = kCols % 64 == 0 ? 64 : kLoad;
#pragma unroll 1
            for (int c = 0; c < kCols; c += kStep) {
                float v[kStep];
#pragma unroll
                for (int h = 0; h < kStep; h += kLoad) {
                    uint32_t b[kLoad];
                    if constexpr (kLoad == 32)
                        EXL3_TMEM_LD32(d + c + h, b);
                    else
                        EXL3_TMEM_LD16(d + c + h, b);
#pragma unroll
                    for (int i = 0; i < kLoad; ++i)
                        v[h + i] = __uint_as_float(b[i]);
                }
                if (c + kStep == kCols)
                    mx_release<CG>(bars, acc);
#pragma unroll
                for (int i = 0; i < kStep; ++i)
                    if (c + i < cols && lane < ch_left)
                        y[(int64_t)(c + i) * p.n + lane] = v[i];
            }
            return true;
        }
    } else if (whole) {
        // everything into registers (16 bits each), so that the MMA issuer
        // gets the accumulator back before the stores
        uint32_t v[kCols / 2];
        if constexpr (kCols % 32 == 0) {
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
                uint32_t b[32];
                EXL3_TMEM_LD32(d + c, b);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[c / 2 + i] = pack2<T>(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
            }
        } else {
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
                uint32_t b[16];
                EXL3_TMEM_LD16(d + c, b);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[c / 2 + i] = pack2<T>(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
            }
        }
        mx_release<CG>(bars, acc);
        if (wide && cols == kCols && ch_left >= 32) {
            // Pairs: the stores are spread over about a third of the next tile's
            // main loop; in one burst they held up its scales' loads (4096 x 4096
            // x 14336: 117 us, without pauses 123).
            const bool pace = CG == 2 && sched.KB >= 4 && seg + 1 < sched.segs;
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
                mx_store8<T, true>(y + (int64_t)c * p.n, p.n, v + c / 2, 8, 32, true);
                if (pace)
                    __nanosleep(sched.KB * 12);
            }
            return true;
        }
#pragma unroll
        for (int c = 0; c < kCols; c += 8)
            if (c < cols)
                mx_store8<T>(y + (int64_t)c * p.n, p.n, v + c / 2, cols - c, ch_left, wide);
        return true;
    }

    // A split tile: fp32 partials to the workspace, [4 columns][lane][4]
    const uint32_t split = g.t - sched.split0;
    uint32_t c_lo;
    int nseg;
    mx_workers(sched, split, c_lo, nseg);
    constexpr size_t kSlot = (size_t)TN * kMxBM;
    const size_t lane_at = (size_t)(c0 / 4) * (4 * kMxBM) + (size_t)(quarter * 32 + lane) * 4;
    float *const mine = p.partials + ((size_t)mx_slot(sched, sched.worker, split) * CG + rank) * kSlot + lane_at;
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
        uint32_t b[16];
        EXL3_TMEM_LD16(d + c, b);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (c + 4 * g < cols)
                __stcg(reinterpret_cast<float4 *>(mine + (size_t)(c / 4 + g) * (4 * kMxBM)),
                       make_float4(__uint_as_float(b[4 * g]), __uint_as_float(b[4 * g + 1]),
                                   __uint_as_float(b[4 * g + 2]), __uint_as_float(b[4 * g + 3])));
    }
    mx_epi_sync<TN, CG>();
    if (threadIdx.x == 32 * kMxEpiWarp0) {
        // the barrier orders the other threads' partials before this fence
        __threadfence();
        uint32_t *counter = &p.counters[split * CG + rank];
        const int last = atomicAdd(counter, 1u) == (uint32_t)(nseg - 1);
        if (last)
            *counter = 0u;  // every segment has arrived: re-arm for the next call
        bars.ticket = last;
        __threadfence();
    }
    __syncwarp();
    mx_epi_sync<TN, CG>();
    if (bars.ticket) {
        // sums in segment order, this CTA's own from TMEM; kAhead segments'
        // loads of 16 columns in flight
        constexpr int kAhead = TN > 128 ? 2 : 4;  // (4 spilled the registers of whole tiles)
        const int own = (int)(sched.worker - c_lo);
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
            uint32_t b[16];
            EXL3_TMEM_LD16(d + c, b);
            float s[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = 0.f;
#pragma unroll 1
            for (int j0 = 0; j0 < nseg; j0 += kAhead) {
                float4 q[kAhead][4];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    if (j0 + j < nseg && j0 + j != own) {
                        const float *src = p.partials +
                                           ((size_t)mx_slot(sched, c_lo + j0 + j, split) * CG + rank) * kSlot + lane_at +
                                           (size_t)(c / 4) * (4 * kMxBM);
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            if (c + 4 * g < cols)
                                q[j][g] = __ldcg(reinterpret_cast<const float4 *>(src + (size_t)g * (4 * kMxBM)));
                    }
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    if (j0 + j < nseg) {
                        const bool o = j0 + j == own;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            s[4 * g] += o ? __uint_as_float(b[4 * g]) : q[j][g].x;
                            s[4 * g + 1] += o ? __uint_as_float(b[4 * g + 1]) : q[j][g].y;
                            s[4 * g + 2] += o ? __uint_as_float(b[4 * g + 2]) : q[j][g].z;
                            s[4 * g + 3] += o ? __uint_as_float(b[4 * g + 3]) : q[j][g].w;
                        }
                    }
                }
            }
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < cols && lane < ch_left)
                        y[(int64_t)(c + i) * p.n + lane] = s[i];
            } else {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = pack2<T>(s[2 * i], s[2 * i + 1]);
#pragma unroll
                for (int h = 0; h < 16; h += 8)
                    if (c + h < cols)
                        mx_store8<T>(y + (int64_t)(c + h) * p.n, p.n, v + h / 2, cols - c - h, ch_left, wide);
            }
        }
    }
    mx_release<CG>(bars, acc);
    return true;
}

// --------------------------------------------------------- main kernel ---

// FUSE: the tokens (kMxFuseRows at most) come as rows of T, and kMxQuantWarps
// warps in turn (one of them in the place of the warp that would deal out the
// tokens' scales) quantise them, codes and scales, straight into the stage: 4
// lanes a rotation, 16 a token and unit, so one pass of a warp a unit (and part of
// k).  Every CTA repeats it for its units, and a launch and its 3 us are gone.  One
// token, k x n, one warp / four (us): 4096 x 4096 10.4 / 9.6, 14336 x 4096 15.1 /
// 12.2, 8192 x 28672 34.3 / 26.6.
// FOLD: 2^p.fold parts of k side by side (mx_split).
template <typename T, int TN, int CG, bool FUSE, bool FOLD>
__global__ void __launch_bounds__(FUSE ? MxTile<TN, CG>::kFuseThreads : MxTile<TN, CG>::kThreads, 1)
    mx4_gemm_kernel(const MxParams p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap)
{
    using S = MxTile<TN, CG>;
    constexpr int ST = S::kStages;
    constexpr int kThreads = FUSE ? S::kFuseThreads : S::kThreads;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    MxBars &bars = *reinterpret_cast<MxBars *>(smem);
    unsigned char *aring = smem + 1024;
    unsigned char *bring = aring + ST * kMxABytes;
    unsigned char *scales = bring + ST * S::kBBytes;
    uint32_t *first = reinterpret_cast<uint32_t *>(scales + ST * S::kScaleBytes);  // [experts + 1] tiles
    uint32_t *frow = first + p.experts + 1;                                          // [experts + 1] rows
    const MxTables tab{first, frow, p.experts};

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int fold = FOLD ? p.fold : 0;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();
    const uint32_t worker = blockIdx.x / CG;
    // Without experts the tiles are known at once, and the warp that issues the
    // copies waits for nobody: it sets up the barriers and begins the first stages
    // while the others set up.  What it reads before grid_dep_wait are weights
    // alone.
    const uint32_t nts = (uint32_t)((p.n + p.bm * CG - 1) / (p.bm * CG));
    const uint32_t tts = (uint32_t)((p.rows + TN - 1) / TN);  // without experts
    const bool early = CG == 1 && !p.offsets;
    const bool ahead = early && warp == kMxTmaWarp;
    if (threadIdx.x == 32 * kMxTmaWarp) {
        for (int s = 0; s < ST; ++s) {
            // the bytes, each CTA's scale warps; or the weights' and each part of the tokens
            mbar_init(&bars.full[s], FUSE ? 2 + (1 << fold) : 1 + CG * 2);
            mbar_init(&bars.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.acc_full[b], 1);
            mbar_init(&bars.acc_empty[b], S::kEpiWarps * CG);
        }
        mbar_init(&bars.drain, 1);
        bars.epi_abort = 0;
        bars.ticket = 0;
        bars.failed = 0;
        for (int r = 0; r < kMxRoles; ++r)
            bars.steps[r] = 0;
        if (early) {
            first[0] = 0;
            first[1] = nts * tts;
            frow[0] = 0;
            frow[1] = (uint32_t)p.rows;
        }
        fence_mbar_init();
    }
    if (ahead) {
        __syncwarp();
        asm volatile("barrier.cta.arrive 2, %0;\n" ::"n"(kThreads) : "memory");
    } else {
        if (warp == kMxMmaWarp)
            mx_tmem_alloc<CG>(&bars.tmem_slot);
        grid_dep_wait();
        grid_dep_launch();
        if (warp == kMxMmaWarp && !early) {
            // prefix sums of the experts' tiles; rows that do not decrease
            uint32_t run = 0, high = 0;
            for (int e0 = 0; e0 <= p.experts; e0 += 32) {
                const int e = e0 + lane;
                uint32_t r = 0;
                if (e <= p.experts)
                    r = p.offsets ? mx_row(p, e) : (e ? (uint32_t)p.rows : 0u);
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, r, d);
                    r = lane >= d && o > r ? o : r;
                }
                r = r > high ? r : high;
                uint32_t before = __shfl_up_sync(0xffffffffu, r, 1);
                before = lane ? before : high;
                // tiles of expert e - 1, whose rows end at r
                const uint32_t v = e >= 1 && e <= p.experts ? (r - before + TN - 1) / TN * nts : 0;
                uint32_t incl = v;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
                    incl += lane >= d ? o : 0;
                }
                if (e <= p.experts) {
                    first[e] = run + incl;
                    frow[e] = r;
                }
                run += __shfl_sync(0xffffffffu, incl, 31);
                high = __shfl_sync(0xffffffffu, r, 31);
            }
        }
        tc_fence_before();
        asm volatile("barrier.cta.sync 2, %0;\n" ::"n"(kThreads) : "memory");
        if constexpr (CG == 2)
            cluster_sync();  // the other CTA's barriers are ready
        tc_fence_after();
    }
    const int KB = p.kb_count;
    const MxSched sched = mx_schedule(early ? nts * tts : first[p.experts], (uint32_t)KB, gridDim.x / CG, worker, p.most);

    if (warp == kMxMmaWarp) {
        if (rank == 0 && sched.segs > 0) {
            // ------------------------------------------------ MMA issuer ---
            const uint32_t base = __shfl_sync(0xffffffffu, bars.tmem_slot, 0);
            const uint32_t a_base = __shfl_sync(0xffffffffu, smem_addr(aring), 0);
            const uint32_t b_base = a_base + ST * kMxABytes, s_base = b_base + ST * S::kBBytes;
            int s = 0;
            uint32_t par = 0;
            bool ok = true;
            bool ready = mbar_try_wait(&bars.full[0], 0);
            for (int seg = 0; seg < sched.segs && ok; ++seg) {
                const MxSeg g = mx_seg(sched, seg);
                const int acc = seg % S::kAcc;
                const uint32_t d = base + (uint32_t)(acc * S::kAccCols);
                if (seg >= S::kAcc)
                    ok = warp_wait_uniform(&bars.acc_empty[acc], (uint32_t)(seg / S::kAcc - 1) & 1u, p.wait_ns);
                for (int kb = g.k0; kb < g.k1 && ok; ++kb) {
                    if (!__all_sync(0xffffffffu, ready))
                        ok = warp_wait_uniform(&bars.full[s], par, p.wait_ns);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t tsa = base + (uint32_t)(S::kAcc * S::kAccCols + s * S::kScaleCols);
                    const uint32_t tsb = tsa + 16;
                    const uint32_t sc = s_base + (uint32_t)(s * S::kScaleBytes);
                    const uint64_t adesc = smem_desc(a_base + (uint32_t)(s * kMxABytes), 16, 1024);
                    const uint64_t bdesc = smem_desc(b_base + (uint32_t)(s * S::kBBytes), 16, 1024);
                    const int left = p.k - kb * kMxBK;
                    // 64 columns per MMA; none behind k, where all parts end there
                    const int steps = left >= kMxBK || fold ? 8 : (left + 63) / 64;
                    uint64_t *const done = &bars.empty[s];
                    if (elect_one()) {
                        // chunk c's scales: weights at tsa + 4c, tokens at tsb + 4 groups c
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_copy_scales<CG>(tsa + 4 * c, sc + 512 * c);
#pragma unroll
                            for (int h = 0; h < S::kBGroups; ++h)
                                tmem_copy_scales<CG>(tsb + 4 * (c * S::kBGroups + h),
                                                     sc + 2048 + 512 * (c * S::kBGroups + h));
                        }
                        // 64 columns are 32 bytes: 2 in the descriptors' address
                        // field; the second box lies behind the first
                        auto mma = [&](int j, uint32_t add) {
                            const uint64_t at = 2 * (j & 3);
                            mma_mxf4<CG>(d, adesc + at + (j >> 2) * (kMxABytes / 2 / 16),
                                         bdesc + at + (j >> 2) * (S::kBBytes / 2 / 16),
                                         (j & 1) ? mx_idesc<TN, CG>(1) : mx_idesc<TN, CG>(0), tsa + 4 * (j >> 1),
                                         tsb + 4 * S::kBGroups * (j >> 1), add);
                        };
                        mma(0, kb > g.k0 ? 1u : 0u);
                        if (steps == 8) {
#pragma unroll
                            for (int j = 1; j < 8; ++j)
                                mma(j, 1u);
                        } else {
#pragma unroll
                            for (int j = 1; j < 7; ++j)
                                if (j < steps)
                                    mma(j, 1u);
                        }
                        mx_commit<CG>(done);
                        if (kb + 1 == g.k1)
                            mx_commit<CG>(&bars.acc_full[acc]);
                    }
                    if (++s == ST) {
                        s = 0;
                        par ^= 1u;
                    }
                    ready = (kb + 1 < g.k1 || seg + 1 < sched.segs) && mbar_try_wait(&bars.full[s], par);
                }
            }
            // no MMA may still be writing TMEM when the CTA tears down
            __syncwarp();
            if (elect_one())
                mx_commit<CG>(&bars.drain);
            __syncwarp();
            ok = warp_wait_uniform(&bars.drain, 0, kDefaultWaitNs) && ok;
            if (!ok && lane == 0)
                mx_failed<CG>(bars, p.status);
        }
    } else if (FUSE && (warp == kMxScaleWarp0 + 1 || warp >= S::kWarps)) {
        // ----------------------------------- quantising a token or two ---
        // Lane: block `lane & 3` of 32 columns of the unit's 128-column group
        // (lane >> 2) & 3 of token lane >> 4.  The worker's units (of each part of
        // k) go round the kMxQuantWarps warps: one alone took 0.95 us a unit, more than its
        // weights' bytes do.
        const int l = lane & 3, grp = (lane >> 2) & 3, row = lane >> 4;
        const int turn = warp >= S::kWarps ? warp - S::kWarps + 1 : 0;
        const bool mine = row < (int)p.rows;
        const T *const xr = (const T *)p.x + (int64_t)(mine ? row : 0) * p.k;
        int s = 0, who = 0;
        uint32_t round = 0;
        bool ok = true;
        for (int seg = 0; seg < sched.segs && ok; ++seg) {
            const MxSeg g = mx_seg(sched, seg);
            for (int kb = g.k0; kb < g.k1 && ok; ++kb) {
                for (int j = 0; j < 1 << fold; ++j) {
                    const bool my_turn = who == turn;
                    if (++who == kMxQuantWarps)
                        who = 0;
                    if (!my_turn)
                        continue;
                    const int col = (kb + j * KB) * kMxBK + 128 * grp + 32 * l;
                    const bool there = col < p.k;  // with the rotation k ends with a group of 128
                    const int at = there ? col : 32 * l < p.k ? 32 * l : 0;
                    int byte = 0;
                    uint4 code;
                    if (p.rotate)
                        code = quantize_block_rotated<T, true>(xr + at, p.signs ? p.signs + at : nullptr, &byte);
                    else
                        code = quantize_block<T>(xr + at, p.signs ? p.signs + at : nullptr, &byte);
                    if (!there) {
                        code = make_uint4(0u, 0u, 0u, 0u);
                        byte = 0;
                    }
                    ok = warp_wait_uniform(&bars.empty[s], (round & 1u) ^ 1u, p.wait_ns);
                    if (!ok)
                        break;
                    if (mine) {
                        // row `at_row` of the box of columns 256 (grp / 2) on, 16-byte
                        // chunk 4 (grp % 2) + l, at the place the swizzle gives it
                        const int chunk = 4 * (grp & 1) + l, at_row = j * (TN >> fold) + row;
                        *reinterpret_cast<uint4 *>(bring + s * S::kBBytes + (grp >> 1) * (S::kBBytes / 2) + at_row * 128 +
                                                   ((chunk ^ (at_row & 7)) << 4)) = code;
                        scales[s * S::kScaleBytes + 2048 + 512 * grp + at_row * 16 + l] = (unsigned char)byte;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars.full[s]);
                }
                if (++s == ST) {
                    s = 0;
                    ++round;
                }
            }
        }
        if (!ok && lane == 0)
            record_timeout(p.status);
    } else if (warp == kMxTmaWarp) {
        // ---------------------------------------------------- producer ---
        // Copies of the codes; both CTAs' bytes of a stage count on the
        // leader's barrier.
        int s = 0;
        int pre = 0;  // stages begun early
        if (ahead) {
            // lane l begins stage l with this worker's unit l
            int seg0 = 0, unit = lane;
            while (seg0 < sched.segs) {
                const MxSeg g = mx_seg(sched, seg0);
                if (unit < g.k1 - g.k0)
                    break;
                unit -= g.k1 - g.k0;
                ++seg0;
            }
            const bool mine = lane < ST && seg0 < sched.segs;
            int col = 0, row = 0;
            if (mine) {
                const MxSeg g = mx_seg(sched, seg0);
                const MxPlace w = mx_place<TN, CG>(p, tab, g.t);
                col = (g.k0 + unit) * (kMxBK / 2);
                row = (int)w.row;
                mbar_arrive_expect_tx(&bars.full[lane], ((p.bm * (kMxBK / 2)) << fold) + (FUSE ? 0 : S::kBBytes));
                for (int h = 0; h < 2; ++h)
                    for (int j = 0; j < 1 << fold; ++j)
                        tma_load_2d<CG>(aring + lane * kMxABytes + h * (kMxABytes / 2) + j * (kMxABytes / 2 >> fold), &wmap,
                                        col + h * (kMxBoxK / 2) + j * KB * (kMxBK / 2), (int)w.wrow,
                                        smem_addr(&bars.full[lane]));
            }
            pre = __popc(__ballot_sync(0xffffffffu, mine));
            grid_dep_wait();
            grid_dep_launch();
            if (mine && !FUSE)
                for (int h = 0; h < 2; ++h)
                    for (int j = 0; j < 1 << fold; ++j)
                        tma_load_2d<CG>(bring + lane * S::kBBytes + h * (S::kBBytes / 2) + j * (S::kBBytes / 2 >> fold), &xmap,
                                        col + h * (kMxBoxK / 2) + j * KB * (kMxBK / 2), row, smem_addr(&bars.full[lane]));
        }
        uint32_t round = 0;                  // of the ring
        uint32_t issued = (1u << pre) - 1u;  // stages that were ever filled: bits
        bool ok = true;
        for (int seg = 0; seg < sched.segs && ok; ++seg) {
            const MxSeg g = mx_seg(sched, seg);
            const MxPlace w = mx_place<TN, CG>(p, tab, g.t);
            const int wrow = (int)w.wrow + (int)rank * kMxBM, xrow = (int)w.row + (int)rank * S::kBRows;
            for (int kb = g.k0; kb < g.k1; ++kb) {
                if (pre > 0) {
                    --pre;
                } else {
                    ok = warp_wait_uniform(&bars.empty[s], (round & 1u) ^ 1u, p.wait_ns);
                    if (!ok)
                        break;
                    const uint32_t bar = CG == 1 ? smem_addr(&bars.full[s]) : leader_addr(&bars.full[s]);
                    if (elect_one()) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&bars.full[s],
                                                  CG * (((p.bm * (kMxBK / 2)) << fold) + (FUSE ? 0 : S::kBBytes)));
                        for (int j = 0; j < 1 << fold; ++j) {
                            unsigned char *const a = aring + s * kMxABytes + j * (kMxABytes / 2 >> fold);
                            unsigned char *const b = bring + s * S::kBBytes + j * (S::kBBytes / 2 >> fold);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int col = (kb + j * KB) * (kMxBK / 2) + h * (kMxBoxK / 2);
                                tma_load_2d<CG>(a + h * (kMxABytes / 2), &wmap, col, wrow, bar);
                                if constexpr (!FUSE)
                                    tma_load_2d<CG>(b + h * (S::kBBytes / 2), &xmap, col, xrow, bar);
                            }
                        }
                    }
                    __syncwarp();
                    issued |= 1u << s;
                }
                if (++s == ST) {
                    s = 0;
                    ++round;
                }
            }
        }
        // Copies in flight end before the CTA does.  Stage st was last filled in
        // this round, or, from s on, in the one before (in round 0: early).
        auto filled = [&](int st) { return st < s || round == 0 ? round : round - 1; };
        if constexpr (CG == 1) {
            // If arrivals are missing, the limit that the first wait runs out of is
            // long enough for all of them.  (The MMAs and their arrivals: the issuer.)
            bool landed = true;
            for (int j = 0; j < ST && landed; ++j) {
                const int st = s + j < ST ? s + j : s + j - ST;
                if (issued >> st & 1u)
                    landed = warp_wait_uniform(&bars.full[st], filled(st) & 1u, kDefaultWaitNs);
            }
            ok = ok && landed;
        } else {
            // Each CTA waits until the MMAs have read its every fill, and so all
            // copies of the pair have landed and the arrivals on `empty` have come.
            // After a timeout the copies are waited for behind the closing barrier.
            for (int st = 0; st < ST && ok; ++st)
                if (issued >> st & 1u)
                    ok = warp_wait_uniform(&bars.empty[st], filled(st) & 1u, p.wait_ns);
            mx_role_done(bars, (int)rank, round * ST + (uint32_t)s);
        }
        if (!ok && lane == 0)
            mx_failed<CG>(bars, p.status);
    } else if (warp < kMxEpiWarp0) {
        // ------------------------------------------------------ scales ---
        // Lane l of the first warp owns the weights' rows l, l + 32, l + 64 and
        // l + 96, of the second the tokens' (of the first 128).  Their scales of
        // 128 columns are the 16 bytes at 16 l of the layout that the tensor
        // core wants: one conflict-free store.  With 256 tokens each warp also
        // takes two of the second 128's four rows, 8 bytes each.  A unit's 16
        // scales of each row are loaded up to kDepth units ahead.  (The warp
        // that issues the copies does nothing else: with a share of this work,
        // 1400 cycles a unit, it was what the MMAs waited for.)
        constexpr int NR = S::kScaleRows;
        const int half = warp - kMxScaleWarp0;  // 0: weights
        const int kblocks = p.k / kMx4Block;
        // load side: segment, unit and rows of the next step
        int fseg = 0, fkb = 0, fend = 0;
        const uint8_t *from = nullptr, *from2 = nullptr;  // scales of rows `lane` and 128 + 64 half + lane
        int have = 0, have2 = 0;                          // rows from there on that exist
        // the part of k of row lane + 32 j
        auto part_of = [&](int j) { return half ? (lane & 15) >> (4 - fold) : j >> (2 - fold); };
        auto enter = [&]() {
            if (fseg < sched.segs) {
                const MxSeg g = mx_seg(sched, fseg);
                const MxPlace w = mx_place<TN, CG>(p, tab, g.t);
                fkb = g.k0;
                fend = g.k1;
                const int64_t tokens = w.row_end - w.row < TN ? w.row_end - w.row : TN;
                const int ch = w.ch + (int)rank * kMxBM;
                const int channels = p.n - ch < p.bm ? p.n - ch : p.bm;
                // (row of a token: lane, in a part's rows)
                const int mine = half && FOLD ? lane & ((16 >> fold) - 1) : lane;
                have = half && FOLD && lane >= 16 ? 0 : (half ? (int)tokens : channels) - mine;
                from = half ? p.xs + (w.row + mine) * p.stride : p.ws + (w.wrow + (ch - w.ch) + lane) * p.stride;
                if constexpr (NR > 4) {
                    have2 = (int)tokens - 128 - 64 * half - lane;
                    from2 = p.xs + (w.row + 128 + 64 * half + lane) * p.stride;
                }
            }
        };
        enter();
        auto fetch = [&](uint4 (&q)[NR]) {
            if (fseg >= sched.segs)
                return;
            const int64_t col = (int64_t)fkb * 16, hop = (int64_t)32 * p.stride;
            if constexpr (FOLD) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int part = part_of(j), rows = half ? 32 * j : 32 * (j & ((4 >> fold) - 1));
                    q[j] = rows < have && 16 * (fkb + part * KB) < p.stride
                               ? *reinterpret_cast<const uint4 *>(from + col + (int64_t)part * KB * 16 + (int64_t)rows * p.stride)
                               : make_uint4(0u, 0u, 0u, 0u);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = 32 * j < have ? *reinterpret_cast<const uint4 *>(from + col + j * hop) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 4; j < NR; ++j)
                q[j] = 32 * (j - 4) < have2 ? *reinterpret_cast<const uint4 *>(from2 + col + (j - 4) * hop)
                                            : make_uint4(0u, 0u, 0u, 0u);
            if (++fkb == fend) {
                ++fseg;
                enter();
            }
        };
        uint4 q[S::kDepth][NR];
#pragma unroll
        for (int d = 0; d < S::kDepth; ++d)
            fetch(q[d]);
        int s = 0, seg = 0, kb = 0, end = 0;
        auto next = [&]() {
            if (seg < sched.segs) {
                const MxSeg g = mx_seg(sched, seg);
                kb = g.k0;
                end = g.k1;
            }
        };
        next();
        uint32_t par = 1;
        uint32_t steps = 0;
        bool ok = true;
        while (seg < sched.segs && ok) {
#pragma unroll
            for (int d = 0; d < S::kDepth; ++d) {
                if (seg < sched.segs && ok) {
                    ok = warp_wait_uniform(&bars.empty[s], par, p.wait_ns);
                    if (ok) {
                        unsigned char *sc = scales + s * S::kScaleBytes + lane * 16;
                        unsigned char *main = sc + (half ? 2048 : 0);
                        const int step = half ? 512 * S::kBGroups : 512;
                        const int last = FOLD ? kb + ((1 << fold) - 1) * KB : kb;
                        const int left = kblocks - last * (kMxBK / kMx4Block);  // scales that exist from this unit on
                        uint32_t v[4][NR];                                    // [128 columns][row]
#pragma unroll
                        for (int j = 0; j < NR; ++j) {
                            v[0][j] = q[d][j].x;
                            v[1][j] = q[d][j].y;
                            v[2][j] = q[d][j].z;
                            v[3][j] = q[d][j].w;
                        }
                        if (left < kMxBK / kMx4Block) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
#pragma unroll
                                for (int j = 0; j < NR; ++j) {
                                    const int at = FOLD ? kb + part_of(j) * KB : kb;
                                    const int n4 = kblocks - at * (kMxBK / kMx4Block) - 4 * c;
                                    v[c][j] &= n4 >= 4 ? 0xffffffffu : (n4 <= 0 ? 0u : (1u << (8 * n4)) - 1u);
                                }
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            *reinterpret_cast<uint4 *>(main + c * step) = make_uint4(v[c][0], v[c][1], v[c][2], v[c][3]);
                            if constexpr (NR > 4)
                                *reinterpret_cast<uint2 *>(sc + 2048 + 512 * (2 * c + 1) + 8 * half) = make_uint2(v[c][4], v[c][5]);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (CG == 1)
                                mbar_arrive(&bars.full[s]);
                            else
                                mbar_arrive_leader(&bars.full[s]);
                        }
                        ++steps;
                        if (++s == ST) {
                            s = 0;
                            par ^= 1u;
                        }
                        if (++kb == end) {
                            ++seg;
                            next();
                        }
                    }
                    // two units at a time: their 16 bytes of a row are one
                    // 32-byte sector, which then crosses from L2 once
                    if (d & 1) {
                        fetch(q[d - 1]);
                        fetch(q[d]);
                    }
                }
            }
        }
        if constexpr (CG == 2)
            mx_role_done(bars, 2 + 2 * (int)rank + half, steps);
        if (!ok && lane == 0)
            mx_failed<CG>(bars, p.status);
    } else {
        // ---------------------------------------------------- epilogue ---
        for (int seg = 0; seg < sched.segs; ++seg)
            if (!mx_epilogue<T, TN, CG, FOLD>(p, bars, tab, sched, bars.tmem_slot, seg, rank))
                break;
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) {
        // The roles of both CTAs have ended, and with them the MMAs (the leader
        // waited for them), the stores and arrivals from one CTA in the other.
        cluster_sync();
        if (*(volatile int *)&bars.failed) {  // the same in both
            if (rank == 0 && warp == kMxTmaWarp)
                mx_settle_pair(bars, ST, kMxABytes + S::kBBytes);
            cluster_sync();
        }
        // The last commit also arrives here, and with it every one before it.
        if (rank == 1 && warp == kMxMmaWarp && sched.segs > 0 && !warp_wait_uniform(&bars.drain, 0, kDefaultWaitNs) && lane == 0)
            record_timeout(p.status);
        __syncwarp();
    }
    if (warp == kMxMmaWarp) {
        tc_fence_after();
        mx_tmem_dealloc<CG>(bars.tmem_slot);
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
    const cuuint32_t boxes[2] = {kMxBoxK / 2, (cuuint32_t)box};
    const cuuint32_t steps[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)codes, dims, strides, boxes, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Token tile for `rows` rows over `experts` experts: the narrowest of 16 .. 128
// that takes an average expert's in one tile.  Above that, 256 tokens x 256
// channels on a pair of CTAs move the fewest bytes per product (1.8 against 1.5
// 128 x 128 x 512 products per SM and us), but leave pairs idle or split where
// tiles are few; from two tiles a pair on they win (us, 128 wide / 256 wide):
// 2048 x 8192 x 8192 (3.5 tiles a pair) 81 / 72, 2048 x 8192 x 28672 262 / 219;
// 2048 x 2048 x 8192 (0.9) 34 / 42, 333 x 4000 x 10001 (1.1) 25 / 34.
static int mx_token_tile(int64_t rows, int64_t n, int64_t experts)
{
    const int64_t each = (rows + experts - 1) / experts;
    if (each <= 128)
        return each <= 16 ? 16 : each <= 32 ? 32 : each <= 64 ? 64 : 128;
    const int64_t tiles = (rows + 255) / 256 * ((n + 255) / 256);
    return tiles >= num_sms() ? 256 : 128;
}

// Workers that may share a tile of kb units: w of them take kb/w units each and
// then w partial sums of TN x 128 per CTA to add, so w = sqrt(kb unit/partial).
// A unit takes 1.1 us (256 tokens), 0.7 us (fewer), a partial written and read
// 0.35 us and 0.012 us a token.  (333 x 4000 x 10001 on pairs took 44 us with 8
// workers on each of the 6 tiles left over, with 1 or 2 it took 32.)
static uint32_t mx_most_workers(int tn, int kb)
{
    const double unit = tn > 128 ? 1.1 : 0.7, partial = 0.35 + 0.012 * tn;
    const double w = sqrt(kb * unit / partial);
    return w < 1.0 ? 1u : (uint32_t)w;
}

// Channels of a CTA's tile, log2 of the parts of k in it, and the workers that may
// share a tile.
struct MxSplit {
    int bm;
    int fold;
    uint32_t most;
};

// Three ways, by the time that each should take (us, without what all have):
// - tiles of 128 channels, some or all split along k over several CTAs: a unit's
//   bytes take 0.77, the sums of split tiles 2 and 0.03 a token;
// - on single CTAs and with one expert, narrower tiles, as many as there are SMs
//   (or that many times 2, 3, ..), each with all of k: nothing to add across CTAs,
//   but a unit of an eighth of the weights still takes 0.5, for its copies,
//   scales and MMAs;
// - for kMxFoldRows tokens, 2 or 4 such narrow tiles' parts of k side by side in
//   one MMA: the channels repeat in the lanes and the tokens in the columns, the
//   sums of part j are where its lanes meet its columns (the rest is not used),
//   and a tile has a half or a quarter of the units.
// Where the product quantises the tokens itself, each CTA does so for its columns
// of k, 0.25 for 512.  (A product of as many rows takes the same way, so that both
// sum in the same order.)
// First / second, us: 16 x 4096 x 4096 8.7 / 8.7 (first), 32 x 4096 x 4096 10.4 / 9.2,
// 64 x 4096 x 4096 12.2 / 9.9, 64 x 4096 x 14336 13.0 / 10.4, 128 x 8192 x 28672 34.7 /
// 31.1, 129 x 8192 x 8192 22.5 / 15.1, 1 x 4096 x 14336 10.0 / 9.4, 1 x 14336 x 4096
// 11.4 / 17.4 (first).  First / third: 1 x 2048 x 2048 7.5 / 5.3, 1 x 4096 x 4096 8.9 /
// 7.1, 1 x 8192 x 8192 11.6 / 10.0; quantising too 8.1 / 6.4, 10.3 / 8.7, 13.0 / 12.9, and 1 x
// 14336 x 4096 12.6 / 16.8 (first).
static MxSplit mx_split(int64_t rows, int64_t n, int kb, int64_t experts, int tn)
{
    MxSplit best = {kMxBM, 0, mx_most_workers(tn, kb)};
    if (experts > 1 || tn > 128 || kb == 1)
        return best;
    const int64_t sms = num_sms(), tts = (rows + tn - 1) / tn;
    const double units = (double)(tts * ((n + kMxBM - 1) / kMxBM) * kb) / (double)sms;
    const double quantise = rows <= kMxFuseRows ? 0.25 : 0.0;
    double time = best.most == 1 ? 1e30 : (0.77 + quantise) * units + 2.0 + 0.03 * tn;
    for (int fold = 0; fold <= 2 && 1 << fold <= kb && (fold == 0 || rows <= kMxFoldRows); ++fold) {
        const int64_t nts = (n + (kMxBM >> fold) - 1) / (kMxBM >> fold);
        const int64_t rounds = (tts * nts + sms - 1) / sms, most = sms * rounds / tts;  // most >= nts
        const int bm = (int)((n + most - 1) / most + 7) / 8 * 8;                         // at most 128 >> fold
        const double unit = 0.006 * (bm << fold) > 0.5 ? 0.006 * (bm << fold) : 0.5;
        const double narrow = unit * (double)(rounds * ((kb + (1 << fold) - 1) >> fold)) + quantise * (double)(rounds * kb);
        if (narrow < time) {
            time = narrow;
            best = MxSplit{bm, fold, 1u};
        }
    }
    return best;
}

static size_t mx_workspace(int64_t rows, int64_t n, int64_t experts)
{
    return kMxSyncArea + (size_t)2 * num_sms() * mx_token_tile(rows, n, experts) * kMxBM * 4;
}

static bool valid_mx_sizes(int64_t m, int64_t k, int64_t n, int64_t experts)
{
    return valid_mx4_k(k) && valid_mx4_rows(m) && n >= 1 && n <= (int64_t)1 << 24 && experts >= 1 &&
           experts <= kMxMaxExperts && experts * n <= (int64_t)1 << 30;
}

template <typename T, int TN, int CG, bool FUSE = false, bool FOLD = false>
static exl3_status launch_mx(const MxParams &p, const CUtensorMap &wmap, const CUtensorMap &xmap, int workers, bool pdl,
                             cudaStream_t s)
{
    using S = MxTile<TN, CG>;
    auto kern = mx4_gemm_kernel<T, TN, CG, FUSE, FOLD>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem + mx_table_bytes(kMxMaxExperts)) !=
        cudaSuccess)
        return EXL3_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(workers * CG));
    cfg.blockDim = dim3(FUSE ? S::kFuseThreads : S::kThreads);
    cfg.dynamicSmemBytes = (size_t)(S::kSmem + mx_table_bytes(p.experts));
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if constexpr (CG == 2) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = 2;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    if (cudaLaunchKernelEx(&cfg, kern, p, wmap, xmap) != cudaSuccess)
        return EXL3_ERR_CUDA;
    return launch_status();
}

template <typename T>
static exl3_status launch_mx_tile(int tn, const MxParams &p, const CUtensorMap &wmap, const CUtensorMap &xmap,
                                  int workers, bool pdl, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2)
        if (p.x)
            return p.fold ? launch_mx<T, 16, 1, true, true>(p, wmap, xmap, workers, pdl, s)
                          : launch_mx<T, 16, 1, true>(p, wmap, xmap, workers, pdl, s);
    if (p.fold)
        return launch_mx<T, 16, 1, false, true>(p, wmap, xmap, workers, pdl, s);
    switch (tn) {
    case 16: return launch_mx<T, 16, 1>(p, wmap, xmap, workers, pdl, s);
    case 32: return launch_mx<T, 32, 1>(p, wmap, xmap, workers, pdl, s);
    case 64: return launch_mx<T, 64, 1>(p, wmap, xmap, workers, pdl, s);
    case 128: return launch_mx<T, 128, 1>(p, wmap, xmap, workers, pdl, s);
    default: return launch_mx<T, 256, 2>(p, wmap, xmap, workers, pdl, s);
    }
}

static exl3_status check_mx(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, const void *y,
                            int dtype, int64_t m, int64_t k, int64_t n, int64_t experts)
{
    if (!valid_mx_sizes(m, k, n, experts) || (dtype != EXL3_F16 && dtype != EXL3_BF16 && dtype != EXL3_F32))
        return EXL3_ERR_INVALID_ARG;
    if (m == 0)
        return EXL3_OK;
    if (!xc || !xs || !wc || !ws || !y || !aligned16(xc) || !aligned16(xs) || !aligned16(wc) || !aligned16(ws) ||
        !aligned16(y))
        return EXL3_ERR_INVALID_ARG;
    const size_t st = (size_t)mx4_scale_stride(k), yb = (size_t)m * (size_t)n * (dtype == EXL3_F32 ? 4 : 2);
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
                          void *workspace, bool pdl, cudaStream_t s, const void *x = nullptr,
                          const void *signs = nullptr, int rotate = 0)
{
    const int tn = mx_token_tile(m, n, experts);
    const int cg = tn > 128 ? 2 : 1;  // CTAs that share a tile
    const int64_t kb_count = (k + kMxBK - 1) / kMxBK;
    const MxSplit split = mx_split(m, n, (int)kb_count, experts, tn);
    const int bm = split.bm;
    CUtensorMap wmap, xmap;
    // (with x the tokens' map is not used)
    if (!code_map(&wmap, wc, experts * n, k / 2, bm) || !code_map(&xmap, x ? wc : xc, x ? n : m, k / 2, (tn / cg) >> split.fold))
        return EXL3_ERR_CUDA;
    MxParams p;
    p.x = x;
    p.signs = (const __half *)signs;
    p.rotate = rotate;
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
    p.kb_count = (int)((kb_count + (1 << split.fold) - 1) >> split.fold);
    p.fold = split.fold;
    p.bm = bm;
    p.experts = (int)experts;
    p.stride = (int)mx4_scale_stride(k);
    p.most = split.most;
    p.wait_ns = wait_limit_ns();
    // units fit 32 bits: at most (rows/TN + experts) tiles of each channel row
    const int64_t tiles =
        ((m + tn - 1) / tn + (experts > 1 ? experts : 0)) * ((n + bm * cg - 1) / (bm * cg));
    if (tiles * p.kb_count >= (int64_t)1 << 31)
        return EXL3_ERR_UNSUPPORTED;
    const int64_t most = num_sms() / cg;
    const int workers = (int)(tiles * p.kb_count < most ? tiles * p.kb_count : most);
    pdl = pdl || (launch_flags() & EXL3_LAUNCH_PDL);
    switch (dtype) {
    case EXL3_F16: return launch_mx_tile<__half>(tn, p, wmap, xmap, workers, pdl, s);
    case EXL3_BF16: return launch_mx_tile<__nv_bfloat16>(tn, p, wmap, xmap, workers, pdl, s);
    default: return launch_mx_tile<float>(tn, p, wmap, xmap, workers, pdl, s);
    }
}

// Workspace of exl3_mx4_linear: the matmul's, then the quantised activations.
struct MxLinearPlan {
    size_t codes, scales, total;
};

static MxLinearPlan mx_linear_plan(int64_t m, int64_t k, int64_t n)
{
    MxLinearPlan pl;
    pl.codes = (mx_workspace(m, n, 1) + 255) / 256 * 256;
    pl.scales = pl.codes + ((size_t)m * (size_t)(k / 2) + 255) / 256 * 256;
    pl.total = pl.scales + (size_t)m * (size_t)mx4_scale_stride(k);
    return pl;
}

}  // namespace exl3

extern "C" size_t exl3_mx4_matmul_workspace_size(int64_t m, int64_t k, int64_t n)
{
    return exl3::valid_mx_sizes(m, k, n, 1) ? exl3::mx_workspace(m, n, 1) : 0;
}

extern "C" exl3_status exl3_mx4_matmul(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws,
                                       void *y, int dtype, int64_t m, int64_t k, int64_t n, void *workspace,
                                       size_t workspace_bytes, void *stream)
{
    using namespace exl3;
    const exl3_status st = check_mx(xc, xs, wc, ws, y, dtype, m, k, n, 1);
    if (st != EXL3_OK || m == 0)
        return st;
    if (!workspace || !aligned16(workspace) || workspace_bytes < mx_workspace(m, n, 1))
        return EXL3_ERR_WORKSPACE;
    return run_mx(xc, xs, nullptr, wc, ws, y, dtype, m, k, n, 1, workspace, false, (cudaStream_t)stream);
}

extern "C" size_t exl3_mx4_matmul_experts_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts)
{
    return exl3::valid_mx_sizes(rows, k, n, experts) ? exl3::mx_workspace(rows, n, experts) : 0;
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
        ranges_overlap(offsets, (size_t)(experts + 1) * 4, y, (size_t)rows * (size_t)n * (dtype == EXL3_F32 ? 4 : 2)))
        return EXL3_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < mx_workspace(rows, n, experts))
        return EXL3_ERR_WORKSPACE;
    return run_mx(xc, xs, offsets, wc, ws, y, dtype, rows, k, n, experts, workspace, false, (cudaStream_t)stream);
}

extern "C" size_t exl3_mx4_linear_workspace_size(int64_t m, int64_t k, int64_t n)
{
    return exl3::valid_mx_sizes(m, k, n, 1) ? exl3::mx_linear_plan(m, k, n).total : 0;
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
    const MxLinearPlan pl = mx_linear_plan(m, k, n);
    const bool fuse = m <= kMxFuseRows;
    if (!workspace || !aligned16(workspace) || workspace_bytes < pl.total)
        return EXL3_ERR_WORKSPACE;
    uint8_t *base = (uint8_t *)workspace;
    uint8_t *xc = base + pl.codes, *xs = base + pl.scales;
    const exl3_status st = check_mx(xc, xs, wc, ws, y, dtype, m, k, n, 1);
    if (st != EXL3_OK)
        return st;
    if (fuse)
        return run_mx(nullptr, nullptr, nullptr, wc, ws, y, dtype, m, k, n, 1, workspace, false, (cudaStream_t)stream, x,
                      signs, rotate);
    const exl3_status q = exl3_mx4_quantize(x, dtype, signs, rotate, nullptr, 1, m, xc, xs, m, k, stream);
    if (q != EXL3_OK)
        return q;
    // launched while the quantiser runs: all but the weights waits for its end
    return run_mx(xc, xs, nullptr, wc, ws, y, dtype, m, k, n, 1, workspace, true, (cudaStream_t)stream);
}
