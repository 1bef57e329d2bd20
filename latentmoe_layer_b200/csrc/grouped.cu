// grouped.cu -- matrix products grouped by expert with ragged sizes, their
// gradients, and the block-scaled 8-bit product (tcgen05, 2-SM pairs).
//
// One engine computes, for every group e (the rows off[e] .. off[e+1] of a
// batch in expert order),
//     out[j, f] = sum_c  B[j, c] A[f, c]
// with f the feature on the MMA's M side (TMEM lanes) and j on its N side:
//
//   GG_FWD  y[r, n]  = sum_k x[r, k]  W[e][n, k]      A = W  (K-major)   B = x  (K-major)
//   GG_DX   dx[r, k] = sum_n dy[r, n] W[e][n, k]      A = W^T (MN-major) B = dy (K-major)
//   GG_DW   dW[e][n, k] = sum_{r in e} dy[r, n] x[r, k]  A = x^T, B = dy^T (both MN-major)
//   GG_FP8  y[r, n] = sum_b sx[r, b] sw[e][n/128, b] sum_{k in block b} xq[r, k] wq[e][n, k]
//   GG_FP8_ROWS  the same with the rows on M and the features on N (epilogue_rows)
//
// Why the features are on M elsewhere. A batch's groups are uneven, and rows on M would
// be padded to 256 per group; the MMA's N takes any multiple of 32, so the
// ragged end of a group costs its own rows only, and a decode batch (a few rows
// per expert) streams each weight tile once with N = 32. The price is a
// transposition of the output, through 2 KB of shared memory per warp (store_rows).
// GG_FP8_ROWS takes large groups, where rounding up to 256 rows costs less than
// one scale per lane gains in the drain.
//
// Why pairs. 128 x 256 tiles on single SMs read 48 KB of operands per 64-deep
// k-block, 96 bytes per SM and cycle at the tensor peak; a pair's 256 x 256 tile
// (tcgen05.mma.cta_group::2) reads 32 KB per SM for the same work.
//
// Structure of one CTA of a pair (one pair per two SMs, persistent over tiles):
//   warp 0       TMA producer (own 128 features of A, own half of B's rows)
//   warp 1       TMEM owner; in the leader CTA, an elected lane issues the MMAs
//   warps 2, 3   8-bit: the products sx * sw of the next four k-blocks, into
//                shared memory; GG_DW: zeros behind a group's last row
//   warps 4-11   epilogue: drain TMEM chunks into fp32 registers, store
// Tiles are found from prefix sums of the counts that every CTA builds in
// shared memory, so a call is one launch and needs no workspace.
//
// Accumulation: TMEM holds a chunk of the contraction (two buffers of 256
// columns), the epilogue adds chunks into fp32 registers while the next one
// runs. The 8-bit forms drain every 128-deep block, where its two scales are applied
// as one fused multiply-add per element (their product is rounded to fp32
// once). fp32 outputs drain every 512, which keeps the tensor core's
// accumulation error near that of fp32 additions; bf16 outputs drain every 4096,
// where that error (2e-5 of a like-signed sum) is still two orders below their rounding.
//
// A group's rows that do not fill a k-block of GG_DW (the contraction runs over
// rows) must not meet the next group's, which may hold anything: warps 2 and 3
// write zeros over those rows of both operands once the k-block has landed.
// Elsewhere rows of a neighbouring group land in output rows that are not
// stored. Features and contraction indices past the matrix are zero-filled by
// the tensor maps.
//
// Every mbarrier wait is bounded (2^24 polls of 4.5 us: 75 s); when one runs out the kernel
// counts it for the host, its cluster waits for its own loads and MMAs, frees TMEM and returns.
#include <cuda_bf16.h>
#include <string.h>

#include <atomic>

#include "grouped.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

constexpr int kGgBN = 256;            // rows (N side) per tile
constexpr int kGgStages = 6;
constexpr int kGgABytes = 128 * 128;  // this CTA's 128 features x 128 bytes
constexpr int kGgBBytes = 128 * 128;  // this CTA's half of the N side
constexpr int kGgThreads = 384;
constexpr int kGgEpiWarps = 8;
constexpr int kGgRaster = 8;          // N-side tiles per raster block (shared weight reads in L2)
constexpr int kScaleBatch = 4;        // k-blocks per batch of scale products
// Registers per thread: 128 x producers' + 256 x epilogue's must not exceed 384 x kLaunchRegs.
// (8-bit: with 56 the scale warps spill, which cost the dense prompt 10%.)
constexpr int kLaunchRegs = 168;
template <int OP>
struct GgRegs {
    static constexpr int kProd = OP >= GG_FP8 ? 72 : 56, kEpi = OP >= GG_FP8 ? 216 : 224;
    static_assert(128 * kProd + 256 * kEpi <= 384 * kLaunchRegs, "register split");
};

struct alignas(1024) GgShared {
    uint8_t a[kGgStages][kGgABytes];
    uint8_t b[kGgStages][kGgBBytes];
    float scale[2][kScaleBatch][kGgBN];
    uint8_t stage[kGgEpiWarps][2048];  // output rows on their way to 16-byte stores
    int off[kMaxE + 2];    // first row of each group, then the end of the last group, then n_rows
    int tiles[kMaxE + 2];  // tile prefix per group
    long long wsum[kGgThreads / 32];
    uint64_t full[kGgStages], empty[kGgStages];
    uint64_t landed[kGgStages], tail[kGgStages];  // GG_DW: a partial k-block is in this CTA's stage; its end is zero
    uint64_t cfull[2], cempty[2], sfull[2], sempty[2], done;
    uint32_t tmem;
    int gave_up;               // a wait of this cluster ran out
    int issued;                // k-blocks this CTA's producer has loaded
    uint32_t sent[kGgStages];  // bytes of a stage's last load that are counted at the leader (partial k-blocks: 0)
};
constexpr size_t kGgSmem = sizeof(GgShared) + 1024;
static_assert(kGgSmem <= 232448, "shared memory");

// Inclusive sum over the block's threads in thread order (called by all threads).
__device__ __forceinline__ long long block_scan(long long v, long long* wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();  // wsum may still be read from an earlier call
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += wsum[w];
    return v;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Row offsets and tile prefixes of all groups. Negative counts count as zero
// and rows past n_rows do not exist, so whatever the counts hold, every row a
// tile touches lies in 0 .. n_rows. With zero_tail the rows behind the last
// group form one more group without a contraction.
template <int OP>
__device__ __forceinline__ int build_groups(const GgParams& P, GgShared& S) {
    const int ft = ceil_div(P.feat, 256);
    const int per = ceil_div(P.n_groups, kGgThreads);
    const int g0 = min(P.n_groups, (int)threadIdx.x * per), g1 = min(P.n_groups, g0 + per);
    long long mine = 0;
    for (int g = g0; g < g1; ++g)
        mine += P.counts ? min(max(ld_global_s32(P.counts + g), 0), P.n_rows) : P.n_rows;
    long long end = block_scan(mine, S.wsum);
    long long at = end - mine;
    long long mt = 0;
    for (int g = g0; g < g1; ++g) {
        const int c = P.counts ? min(max(ld_global_s32(P.counts + g), 0), P.n_rows) : P.n_rows;
        const int lo = (int)min(at, (long long)P.n_rows), hi = (int)min(at + c, (long long)P.n_rows);
        S.off[g] = lo;
        mt += OP == GG_DW ? ceil_div(P.cols, kGgBN) : ceil_div(hi - lo, kGgBN);
        at += c;
        if (g == P.n_groups - 1) S.off[P.n_groups] = hi;
    }
    mt *= ft;
    const long long tend = block_scan(mt, S.wsum);
    long long tat = tend - mt;
    at = end - mine;
    for (int g = g0; g < g1; ++g) {
        const int c = P.counts ? min(max(ld_global_s32(P.counts + g), 0), P.n_rows) : P.n_rows;
        const int lo = (int)min(at, (long long)P.n_rows), hi = (int)min(at + c, (long long)P.n_rows);
        S.tiles[g] = (int)tat;
        tat += (long long)ft * (OP == GG_DW ? ceil_div(P.cols, kGgBN) : ceil_div(hi - lo, kGgBN));
        at += c;
        if (g == P.n_groups - 1) {
            S.tiles[P.n_groups] = (int)tat;
            S.off[P.n_groups + 1] = P.n_rows;
            S.tiles[P.n_groups + 1] = (int)tat + (P.zero_tail ? ft * ceil_div(P.n_rows - hi, kGgBN) : 0);
        }
    }
    __syncthreads();
    return S.tiles[P.n_groups + 1];
}

struct GgTile {
    int e;      // group
    int row0;   // first row of the tile (GG_DW: of the group)
    int col0;   // GG_DW: first dW row (N index) of the tile
    int ncols;  // valid N-side rows of the tile
    int neff;   // the MMA's N: ncols rounded up to 32
    int feat0;  // first feature of the pair
    int kb0;    // first k-block of this pair's share of the contraction
    int nkb;    // k-blocks of the share
    int rem;    // GG_DW: rows of the last k-block when it is partial, else 0
};

// Tile t. Within a group, raster blocks of kGgRaster N-side tiles sweep the
// features, so that the pairs running at once share both operands in L2.
// `e` carries the last tile's group: a CTA's tiles only move forward.
template <int OP>
__device__ __forceinline__ GgTile decode(const GgParams& P, const GgShared& S, int t, int& e, int part, int splits) {
    if (t >= S.tiles[e + 1]) {
        int lo = e + 1, hi = P.n_groups;  // tiles[lo] <= t < tiles[hi + 1]
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (S.tiles[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        e = lo;
    }
    const int ft = ceil_div(P.feat, 256);
    const int local = t - S.tiles[e];
    const int ct = (S.tiles[e + 1] - S.tiles[e]) / ft;
    const int g = local / (kGgRaster * ft), r = local % (kGgRaster * ft);
    const int ms = min(kGgRaster, ct - g * kGgRaster);
    const int c = g * kGgRaster + r % ms;
    const int cnt = S.off[e + 1] - S.off[e];
    // a group's rows are spread evenly over its tiles (in steps of 32): pairs take tiles in
    // turn, so a full tile here and a short one there would leave some pairs waiting
    const int per = OP == GG_DW || OP == GG_FP8_ROWS ? kGgBN : (ceil_div(cnt, ct) + 31) & ~31;
    GgTile ti;
    ti.e = e;
    ti.feat0 = (r / ms) * 256;
    if (OP == GG_DW) {
        ti.row0 = S.off[e];
        ti.col0 = c * kGgBN;
        ti.ncols = min(kGgBN, P.cols - ti.col0);
        ti.kb0 = 0;
        ti.nkb = ceil_div(cnt, 64);
        ti.rem = cnt & 63;
    } else {
        ti.row0 = S.off[e] + c * per;
        ti.col0 = 0;
        ti.ncols = min(per, cnt - c * per);
        const int nkb = e < P.n_groups ? ceil_div(P.cdim, OP == GG_FP8 || OP == GG_FP8_ROWS ? 128 : 64) : 0;
        constexpr int kUnit = OP == GG_FP8 ? kScaleBatch : 1;  // scales are read in batches
        const int units = ceil_div(nkb, kUnit);
        ti.kb0 = units * part / splits * kUnit;
        ti.nkb = min(nkb, units * (part + 1) / splits * kUnit) - ti.kb0;
        ti.rem = 0;
    }
    ti.neff = ((OP == GG_FP8_ROWS ? min(kGgBN, P.feat - ti.feat0) : ti.ncols) + 31) & ~31;
    return ti;
}

// Load whose completion is counted in this CTA (bar: one of its own barriers).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t leader_bar, int x, int y,
                                                 int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// GG_FP8: 128-deep blocks handed to the epilogue at once, side by side in a
// 256-column buffer: a narrow tile's block is over too soon to pay for a hand-over
// of its own. Divides kScaleBatch.
__device__ __forceinline__ int blocks_per_drain(int neff) { return neff <= 64 ? 4 : neff <= 128 ? 2 : 1; }

template <bool kF8>
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (kF8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        umma_bf16_pair(d, a, b, idesc, accumulate);
}

// Arrive on the barrier at this offset in both CTAs of the pair (bits of mask: their
// ranks in the cluster) once the leader's tcgen05 operations so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t mask) {
    asm volatile(
        "{\n\t.reg .b16 m;\n\t"
        "cvt.u16.u32 m, %1;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(mask)
        : "memory");
}

// Operand whose contraction index runs along shared-memory rows (MN-major):
// 64 contraction rows of 128 bytes (64 features) per 8 KB sub-tile, 128-byte
// swizzle; 8-row groups 1024 bytes apart (stride offset), the next 64 features
// 8192 bytes on (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// Gives a buffer of TMEM back (the barrier may be the other CTA's) once the warp's loads
// from it have completed (wait::ld). The fence orders them, so the arrival needs no
// release, which would first wait for the thread's own stores to global memory (1.3K to
// 3.7K cycles per hand-over at cluster scope). Predicated, so that the warp does not branch.
__device__ __forceinline__ void release_tmem(uint32_t cluster_addr, int lane) {
    tc_fence_before();
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr),
        "r"(lane)
        : "memory");
}
// Arrive (where `on`) on this CTA's barrier, with a release: what the warp read from shared
// memory before may be overwritten after it. Predicated too.
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool on) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"((uint32_t)on)
        : "memory");
}

// One lane of a converged warp; the compiler then knows the branch is uniform.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// ---- Bounded waits. One that runs out makes the whole cluster give up (every CTA has the word,
// polled in its own shared memory) and is counted for the host. Other clusters, and other
// launches, go on: the word that the host reads is never read here.
__device__ __forceinline__ void give_up(GgShared& S, const GgParams& P) {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
#pragma unroll 1
    for (uint32_t r = 0; r < n; ++r)
        asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(mapa_shared(&S.gave_up, r)) : "memory");
    atomicAdd(P.err, 1);
}
__device__ __forceinline__ bool gave_up(const GgShared& S) {
    int v;
    asm volatile("ld.relaxed.cluster.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(&S.gave_up)) : "memory");
    return v != 0;
}
// try_wait that acquires at cluster scope: for arrivals of generic accesses in the other CTA.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Wait of one elected thread.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, GgShared& S, const GgParams& P) {
    if (!kCluster && mbar_test_wait(bar, parity)) return true;
    for (unsigned i = 0; i < P.spin; ++i) {
        if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 255u && gave_up(S)) return false;
    }
    give_up(S, P);
    return false;
}
// Wait of a whole warp: all lanes see the phase completed, or all give up. (Lanes that
// decide alone could part at the limit, ahead of a __syncwarp or a TMEM load that needs them all.)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, GgShared& S, const GgParams& P) {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) return true;
    for (unsigned i = 0; i < P.spin; ++i) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 255u && __any_sync(0xFFFFFFFFu, gave_up(S))) return false;
    }
    if ((threadIdx.x & 31) == 0) give_up(S, P);
    __syncwarp();
    return false;
}
// Wait for operations already under way, which end by themselves: does not leave when the
// cluster gives up, and is bounded all the same.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    for (unsigned i = 0; i < (1u << 24); ++i)
        if (mbar_try_wait(bar, parity)) return;
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Zeros the rows from rem to the next multiple of 16 (the MMAs' depth; rows behind
// that are not multiplied) of `subs` sub-tiles of 128-byte rows: 64 threads. Whole
// rows, so the swizzle, which stays inside a row, does not matter.
__device__ __forceinline__ void zero_rows(uint8_t* dst, int subs, int rem, int tid) {
    const int end = ((rem + 15) & ~15) * 8;
    for (int sub = 0; sub < subs; ++sub)
        for (int i = rem * 8 + tid; i < end; i += 64)
            *reinterpret_cast<uint4*>(dst + sub * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// 16 TMEM lanes x 32 columns: register 4 b + 2 s + j holds lane (l / 4) + 8 s, column
// 8 b + 2 (l % 4) + j of thread l.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Waits for the loads so far. Every use of their registers (below) is volatile asm, which
// keeps its order after this one; other code must not touch them.
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// acc += (lo, hi) and acc += (lo, hi) * s for registers that a load has written.
__device__ __forceinline__ void add_loaded(uint64_t& acc, uint32_t lo, uint32_t hi) {
    asm volatile("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tadd.rn.f32x2 %0, %0, v;\n\t}" : "+l"(acc) : "r"(lo), "r"(hi));
}
__device__ __forceinline__ void fma_loaded(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
    asm volatile("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(acc) : "r"(lo), "r"(hi), "l"(s));
}
// Four consecutive k-blocks' scales of one operand row, zero past its `left` last ones.
__device__ __forceinline__ float4 load_scales(const float* p, int left, bool wide) {
    if (wide) {
        const uint4 v = ld_global_v4(p);
        return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
    float4 s = make_float4(ld_global_f32(p), 0.f, 0.f, 0.f);
    if (left > 1) s.y = ld_global_f32(p + 1);
    if (left > 2) s.z = ld_global_f32(p + 2);
    if (left > 3) s.w = ld_global_f32(p + 3);
    return s;
}

// Four 8 x 8 matrices of 16-bit values, transposed on their way to shared memory.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// The warp's accumulators: acc[h][b][s] holds features 16 h + 8 s + l / 4 of the
// warp's 32, columns (output rows) 8 b + 2 (l % 4) and the next one.
typedef uint64_t Acc[2][16][2];

// Stores the warp's 32 features x nv output rows; `out` points at its first feature in
// the first row, `feats` features exist from there. Transposed through 2 KB of
// shared memory (bf16: 32 rows of 64 bytes by stmatrix; fp32: 16 rows of 128 bytes;
// pieces swizzled so that neither side conflicts) into 16-byte stores of whole
// sectors: two-byte stores straight from the registers took 10K cycles per tile.
__device__ __forceinline__ void store_rows(const Acc& acc, uint8_t* stage, void* out, long long ldo, int nv, int feats,
                                           bool f32, int lane) {
    if (f32) {
        float* st = reinterpret_cast<float*>(stage);
#pragma unroll
        for (int rb = 0; rb < 8; ++rb) {
            if (rb * 16 >= nv) break;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float lo, hi;
                        unpack2(acc[h][rb * 2 + b][s], lo, hi);
                        float* p = st + (b * 8 + 2 * (lane & 3)) * 32 + ((h * 16 + s * 8 + (lane >> 2)) ^ ((lane & 3) << 3));
                        p[0] = lo;
                        p[32] = hi;
                    }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (lane >> 3) + 4 * i, f = (lane & 7) * 4;
                const float4 v = *reinterpret_cast<const float4*>(st + row * 32 + (f ^ (((row >> 1) & 3) << 3)));
                if (rb * 16 + row < nv && f < feats)
                    *reinterpret_cast<float4*>(static_cast<float*>(out) + (long long)(rb * 16 + row) * ldo + f) = v;
            }
            __syncwarp();
        }
    } else {
        const uint32_t st = smem_u32(stage);
        const int m = lane >> 3, r8 = lane & 7;
        const uint32_t dst = st + (uint32_t)(r8 * 64 + ((m ^ ((r8 >> 1) & 3)) << 4));
#pragma unroll
        for (int rb = 0; rb < 4; ++rb) {
            if (rb * 32 >= nv) break;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    unpack2(acc[i >> 1][rb * 4 + b][i & 1], lo, hi);
                    v[i] = pack_bf16x2(lo, hi);
                }
                stmatrix_trans(dst + b * 512, v[0], v[1], v[2], v[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (lane >> 2) + 8 * i, f = (lane & 3) * 8;
                const uint4 v = ld_shared_v4(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
                if (rb * 32 + row < nv && f < feats)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + (long long)(rb * 32 + row) * ldo + f) = v;
            }
            __syncwarp();
        }
    }
}

// Adds 32 lanes x 32 NG columns of TMEM to acc, GG_FP8 with a factor per column at sc (the
// thread's first pair of columns); gives the buffer back after the last load of the
// `last` part. bf16 loads run one group ahead of the additions. (NG is a template argument
// because conditions between the groups cost moves of the registers in flight.)
template <int NG, bool kF8>
__device__ __forceinline__ void drain_columns(Acc& acc, uint32_t taddr, const float* sc, bool last, uint32_t release,
                                              int lane) {
    constexpr int kAhead = kF8 ? 0 : 1;  // GG_FP8's tiles mostly have one group, and its registers are full
    uint32_t raw[1 + kAhead][32];
    if (kAhead) {
        tmem_ld_16x32(taddr, &raw[0][0]);
        tmem_ld_16x32(taddr + (16u << 16), &raw[0][16]);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        uint32_t* r = raw[kAhead ? g & 1 : 0];
        if (!kAhead) {
            tmem_ld_16x32(taddr + (uint32_t)(32 * g), r);
            tmem_ld_16x32(taddr + (uint32_t)(32 * g) + (16u << 16), r + 16);
        }
        tmem_ld_wait();
        if (g + 1 < NG) {
            if (kAhead) {
                uint32_t* n = raw[kAhead ? (g + 1) & 1 : 0];
                tmem_ld_16x32(taddr + (uint32_t)(32 * (g + 1)), n);
                tmem_ld_16x32(taddr + (uint32_t)(32 * (g + 1)) + (16u << 16), n + 16);
            }
        } else if (last) {
            release_tmem(release, lane);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint64_t s2 = kF8 ? *reinterpret_cast<const uint64_t*>(sc + 32 * g + 8 * b) : 0ull;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint64_t& a = acc[i >> 1][4 * g + b][i & 1];
                const uint32_t* v = r + 16 * (i >> 1) + 4 * b + 2 * (i & 1);
                if (kF8) fma_loaded(a, v[0], v[1], s2);
                else add_loaded(a, v[0], v[1]);
            }
        }
    }
}

// 32 TMEM lanes x 16 columns: register i holds the thread's lane, column i.
__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Adds s x (32 lanes x 32 NG columns of TMEM) to acc and gives the buffer back when the
// last load has arrived; loads run one group ahead of the additions.
template <int NG>
__device__ __forceinline__ void drain_rows(uint64_t (&acc)[64], uint32_t taddr, float s, uint32_t release, int lane) {
    const uint64_t s2 = pack2(__float_as_uint(s), __float_as_uint(s));
    uint32_t raw[2][32];
    tmem_ld_32x16(taddr, &raw[0][0]);
    tmem_ld_32x16(taddr + 16, &raw[0][16]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        uint32_t* r = raw[g & 1];
        tmem_ld_wait();
        if (g + 1 < NG) {
            tmem_ld_32x16(taddr + (uint32_t)(32 * (g + 1)), &raw[(g + 1) & 1][0]);
            tmem_ld_32x16(taddr + (uint32_t)(32 * (g + 1) + 16), &raw[(g + 1) & 1][16]);
        } else {
            release_tmem(release, lane);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) fma_loaded(acc[16 * g + i], r[2 * i], r[2 * i + 1], s2);
    }
}

// GG_FP8_ROWS: a warp holds 32 rows (a lane each) x 128 features of one weight
// block, so a 128-deep block's factor sx * sw is one register per thread and the
// drain touches no shared memory, whose bandwidth the MMA's operands use up. It reads
// all 128 columns even of a narrower tile: one straight path instead of a choice by
// width took the dense prompt (16384 x 10240 x 8192) from 1504 to 1425 us.
__device__ __forceinline__ void epilogue_rows(const GgParams& P, GgShared& S, int pair, int npairs, int ntiles,
                                              uint32_t rank, int q, int h, int lane, uint32_t tmem_base, uint32_t cempty0) {
    int buf = 0, sbuf = 0, e = 0, stage = 0;
    uint32_t bphase = 0, sphase = 0;
    const bool frees = q == 0 && h == 0 && lane == 0;
    auto free_stage = [&] {  // the block's operands have been read
        mbar_arrive_if(&S.empty[stage], frees);
        if (++stage == kGgStages) stage = 0;
    };
    for (int t = pair; t < ntiles; t += npairs) {
        const GgTile ti = decode<GG_FP8_ROWS>(P, S, t, e, 0, 1);
        const int c0 = h * 128;  // the warp's first column
        uint64_t acc[64];  // columns 2 i and 2 i + 1
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0ull;
        float4 f;
        for (int kb = 0; kb < ti.nkb; ++kb) {
            if (kb % kScaleBatch == 0) {
                if (!wait_warp(&S.sfull[sbuf], sphase, S, P)) return;
                f = *reinterpret_cast<const float4*>(&S.scale[sbuf][0][0] + 4 * (h * 128 + q * 32 + lane));
                __syncwarp();
                mbar_arrive_if(&S.sempty[sbuf], lane == 0);
                if (++sbuf == 2) {
                    sbuf = 0;
                    sphase ^= 1u;
                }
            }
            const float s = f.x;
            f = make_float4(f.y, f.z, f.w, 0.f);
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c0;
            if (!wait_warp(&S.cfull[buf], bphase, S, P)) return;
            free_stage();
            tc_fence_after();
            const uint32_t release = cempty0 + 8u * (uint32_t)buf, at = taddr + (uint32_t)(buf * kGgBN);
            drain_rows<4>(acc, at, s, release, lane);  // columns past the matrix come from earlier blocks and are not stored
            if (++buf == 2) {
                buf = 0;
                bphase ^= 1u;
            }
        }
        // rows of 64 features (bf16) or 32 (fp32), 4 rows x 128 bytes per store through shared memory:
        // the warp's 2 KB hold 16 rows of 128 bytes, pieces swizzled by the row's index modulo 8
        const int nrows = min(32, ti.ncols - ((int)rank * 128 + q * 32));  // may be <= 0
        uint8_t* st = S.stage[q + 4 * h];
        const int esz = P.out_f32 ? 4 : 2, per = 128 / esz;
        char* out = static_cast<char*>(P.out) +
                    ((long long)(ti.row0 + (int)rank * 128 + q * 32) * P.ldo + ti.feat0 + c0) * esz;
        const int feats = P.feat - ti.feat0 - c0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // 128 bytes of every row
            if ((P.out_f32 || g < 2) && g * per < feats) {
#pragma unroll
                for (int hr = 0; hr < 2; ++hr) {  // 16 of the warp's rows
                    if ((lane >> 4) == hr) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint4 v;
                            if (P.out_f32) {
                                float a[4];
                                unpack2(acc[16 * g + 2 * c], a[0], a[1]);
                                unpack2(acc[16 * g + 2 * c + 1], a[2], a[3]);
                                v = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                                               __float_as_uint(a[3]));
                            } else {
                                float a[8];
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    unpack2(acc[32 * (g & 1) + 4 * c + j], a[2 * j], a[2 * j + 1]);
                                v = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                                               pack_bf16x2(a[6], a[7]));
                            }
                            *reinterpret_cast<uint4*>(st + (lane & 15) * 128 + ((c ^ (lane & 7)) << 4)) = v;
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = (lane >> 3) + 4 * i, c = lane & 7;
                        const uint4 v = ld_shared_v4(st + r * 128 + ((c ^ (r & 7)) << 4));
                        if (hr * 16 + r < nrows && g * per + c * (16 / esz) < feats)
                            *reinterpret_cast<uint4*>(out + ((long long)(hr * 16 + r) * P.ldo) * esz + g * 128 + c * 16) = v;
                    }
                    __syncwarp();
                }
            }
        }
    }
}

// A split contraction: the pairs of a cluster each hold a tile's sum over their share.
// The later ones write theirs into the stages of the first pair's CTA of the same
// features (a[0] onwards: hc KB per pair), which adds them in order. Entry i of thread
// t is at (i * 256 + t) * 8, so that a warp's accesses are contiguous.
__device__ __forceinline__ void send_partial(const Acc& acc, uint8_t* stages, int part, uint32_t rank, int hc) {
    const uint32_t to = mapa_shared(stages, rank) + (uint32_t)((part - 1) * hc * 1024 + ((int)threadIdx.x - 128) * 8);
#pragma unroll
    for (int b = 0; b < 16; ++b)
        if (8 * b < hc) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to + (uint32_t)((4 * b + i) * 2048)),
                             "l"(acc[i >> 1][b][i & 1])
                             : "memory");
        }
}
__device__ __forceinline__ void add_partials(Acc& acc, const uint8_t* stages, int splits, int hc) {
    for (int part = 1; part < splits; ++part) {
        const uint8_t* from = stages + (part - 1) * hc * 1024 + ((int)threadIdx.x - 128) * 8;
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (8 * b < hc) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i >> 1][b][i & 1] =
                        add2(acc[i >> 1][b][i & 1], *reinterpret_cast<const uint64_t*>(from + (4 * b + i) * 2048));
            }
    }
}

// How often n k-blocks in turn have used stage s.
__device__ __forceinline__ int uses(int n, int s) { return n > s ? (n - s + kGgStages - 1) / kGgStages : 0; }

// After the cluster gave up: waits for the pair's loads in flight. They are counted on the leader's
// full barriers, each phase of which waits for the bytes of both CTAs; where only one CTA's
// producer got to load a k-block, the other's share is made up here. (A CTA can be at most one
// use of a stage ahead: reusing it takes an MMA that read both CTAs' operands.)
__device__ void drain_loads(GgShared& S, uint32_t other) {
    int theirs;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(theirs) : "r"(mapa_shared(&S.issued, other)) : "memory");
#pragma unroll 1
    for (int s = 0; s < kGgStages; ++s) {
        const int u0 = uses(S.issued, s), u1 = uses(theirs, s);
        uint32_t b1;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(b1) : "r"(mapa_shared(&S.sent[s], other)) : "memory");
        if (u0 > u1 && S.sent[s])
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&S.full[s])), "r"(S.sent[s])
                         : "memory");
        if (u1 > u0) {
            if (b1 == 0) continue;  // a partial k-block: counted in that CTA
            mbar_arrive_expect_tx(&S.full[s], b1);
        }
        const int u = max(u0, u1);
        if (u > 0) drain_wait(&S.full[s], (uint32_t)(u - 1) & 1u);
    }
}

// kSplit: a cluster holds P.splits pairs, which share each tile's contraction. (An
// instantiation of its own: ranks known at compile time keep the others' registers
// free of spills, which cost the 8-bit products 15%.)
template <int OP, bool kSplit>
__global__ void __launch_bounds__(kGgThreads, 1) k_grouped(const __grid_constant__ GgParams P) {
    constexpr bool kF8 = OP == GG_FP8 || OP == GG_FP8_ROWS, kRowsM = OP == GG_FP8_ROWS, kAMN = OP == GG_DX || OP == GG_DW, kBMN = OP == GG_DW;
    extern __shared__ uint8_t smem_raw[];
    GgShared& S = *reinterpret_cast<GgShared*>(smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw)));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // `pair` numbers the clusters
    const uint32_t crank = cluster_ctarank(), rank = kSplit ? crank & 1u : crank, lead = kSplit ? crank & ~1u : 0u;
    const bool leader = rank == 0;
    const int splits = kSplit ? P.splits : 1, part = kSplit ? (int)(crank >> 1) : 0;
    const int pair = (int)blockIdx.x / (2 * splits), npairs = (int)gridDim.x / (2 * splits);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kGgStages; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
            mbar_init(&S.landed[s], 1);
            mbar_init(&S.tail[s], 4);  // two zeroing warps in each CTA
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.cfull[b], 1);
            mbar_init(&S.cempty[b], 2 * kGgEpiWarps);  // both CTAs' epilogue warps
            mbar_init(&S.sfull[b], 2);
            mbar_init(&S.sempty[b], kGgEpiWarps);
        }
        mbar_init(&S.done, 1);
        S.gave_up = 0;
        S.issued = 0;
        fence_mbar_init();
        prefetch_tmap(&P.a_map);
        for (int i = 0; i < (kBMN ? 1 : 4); ++i) prefetch_tmap(&P.b_map[i]);
    }
    dependent_wait_and_release();
    if (warp == 1) {
        tmem_alloc_pair(&S.tmem, 512);
        tmem_relinquish_pair();
    }
    const int ntiles = build_groups<OP>(P, S);
    tc_fence_before();
    cluster_sync_all();  // barriers, TMEM and tables of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem_base = S.tmem;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(GgRegs<OP>::kProd));
        if (warp == 0 && elect_one()) {
            // -------------------------------------------- TMA producer (both CTAs)
            int stage = 0, e = 0;
            int issued = 0;
            uint32_t phase = 0, partial = 0, partial_n = 0;
            const uint32_t full0 = mapa_shared(&S.full[0], lead);
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e, part, splits);
                const int half = ti.neff / 2, f0 = ti.feat0 + (int)rank * 128;
                const int b0 = (kBMN ? ti.col0 : ti.row0) + (int)rank * half;
                const uint32_t bytes_b = kRowsM ? (uint32_t)kGgBBytes : kBMN ? (uint32_t)((half + 63) / 64) * 8192u : (uint32_t)half * 128u;
                for (int kb = 0; kb < ti.nkb; ++kb) {
                    if (!wait_one(&S.empty[stage], phase ^ 1u, S, P)) {
                        ok = false;
                        break;
                    }
                    if (OP == GG_DW && ti.rem && kb == ti.nkb - 1) {
                        // counted in this CTA, whose warps 2 and 3 then zero the rows behind the group
                        const int r = ti.row0 + kb * 64;
                        mbar_arrive_expect_tx(&S.landed[stage], kGgABytes + bytes_b);
                        tma_load_3d(S.a[stage], &P.a_map, &S.landed[stage], f0, r, 0);
                        tma_load_3d(S.a[stage] + 8192, &P.a_map, &S.landed[stage], f0 + 64, r, 0);
                        tma_load_3d(S.b[stage], &P.b_map[0], &S.landed[stage], b0, r, 0);
                        if (half > 64) tma_load_3d(S.b[stage] + 8192, &P.b_map[0], &S.landed[stage], b0 + 64, r, 0);
                        if (leader) mbar_arrive(&S.full[stage]);
                        S.sent[stage] = 0;
                        partial |= 1u << stage;
                        partial_n ^= 1u << stage;
                    } else {
                        if (leader) mbar_arrive_expect_tx(&S.full[stage], 2u * (kGgABytes + bytes_b));
                        const uint32_t bar = full0 + 8u * (uint32_t)stage;
                        if (kRowsM) {
                            tma_load_3d_pair(S.a[stage], &P.b_map[0], bar, kb * 128, ti.row0 + (int)rank * 128, 0);
                            tma_load_3d_pair(S.b[stage], &P.a_map, bar, kb * 128, ti.feat0 + (int)rank * half, ti.e);
                        } else if (OP == GG_FWD || OP == GG_FP8) {
                            tma_load_3d_pair(S.a[stage], &P.a_map, bar, (ti.kb0 + kb) * (kF8 ? 128 : 64), f0, ti.e);
                        } else if (OP == GG_DX) {
                            tma_load_3d_pair(S.a[stage], &P.a_map, bar, f0, (ti.kb0 + kb) * 64, ti.e);
                            tma_load_3d_pair(S.a[stage] + 8192, &P.a_map, bar, f0 + 64, (ti.kb0 + kb) * 64, ti.e);
                        } else {
                            const int r = ti.row0 + kb * 64;
                            tma_load_3d_pair(S.a[stage], &P.a_map, bar, f0, r, 0);
                            tma_load_3d_pair(S.a[stage] + 8192, &P.a_map, bar, f0 + 64, r, 0);
                            tma_load_3d_pair(S.b[stage], &P.b_map[0], bar, b0, r, 0);
                            if (half > 64) tma_load_3d_pair(S.b[stage] + 8192, &P.b_map[0], bar, b0 + 64, r, 0);
                        }
                        if (!kBMN && !kRowsM) {
                            const int x = (ti.kb0 + kb) * (kF8 ? 128 : 64);
                            // half rows in boxes of 128, 64, 32 and 16: few requests, no row too many
                            int r = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (half & (128 >> i)) {
                                    tma_load_3d_pair(S.b[stage] + r * 128, &P.b_map[i], bar, x, b0 + r, 0);
                                    r += 128 >> i;
                                }
                        }
                        S.sent[stage] = kGgABytes + bytes_b;
                    }
                    ++issued;
                    if (++stage == kGgStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            S.issued = issued;
            // every stage given back: its loads have landed and been read, and no arrival at
            // this CTA's barriers is under way when it leaves
            for (int s = 0; s < kGgStages && ok; ++s)
                if (issued > s) ok = wait_one(&S.empty[s], uses(issued, s) - 1 & 1, S, P);
            if (!ok)  // drain_loads does the rest; the stage's last partial block has parity (their number - 1) % 2
                for (int s = 0; s < kGgStages; ++s)
                    if ((partial >> s) & 1u) drain_wait(&S.landed[s], (~partial_n >> s) & 1u);
        } else if (warp == 1 && leader && elect_one()) {
            // -------------------------------------------- MMA issuer (leader only)
            constexpr uint32_t type = kF8 ? 0u : 1u;  // e4m3 : bf16
            constexpr uint32_t idesc0 = (1u << 4) | (type << 7) | (type << 10) | ((kAMN ? 1u : 0u) << 15) |
                                        ((kBMN ? 1u : 0u) << 16) | ((256u >> 4) << 24);
            constexpr uint64_t a_step = kAMN ? 2048 >> 4 : 32 >> 4, b_step = kBMN ? 2048 >> 4 : 32 >> 4;
            int stage = 0, buf = 0, e = 0;
            uint32_t phase = 0, bphase = 0, tphase = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e, part, splits);
                const uint32_t idesc = idesc0 | ((uint32_t)(ti.neff >> 3) << 17);
                const int ck = kRowsM ? 1 : kF8 ? blocks_per_drain(ti.neff) : P.chunk_kb;
                for (int kb0 = 0; kb0 < ti.nkb && ok; kb0 += ck) {
                    if (!wait_one(&S.cempty[buf], bphase ^ 1u, S, P)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t d = tmem_base + (uint32_t)(buf * kGgBN);
                    const int kb1 = min(ti.nkb, kb0 + ck);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!wait_one(&S.full[stage], phase, S, P)) {
                            ok = false;
                            break;
                        }
                        int steps = 4;
                        if (OP == GG_DW && ti.rem && kb == ti.nkb - 1) {
                            steps = (ti.rem + 15) >> 4;
                            if (!wait_one<true>(&S.tail[stage], (tphase >> stage) & 1u, S, P)) {
                                ok = false;
                                break;
                            }
                            tphase ^= 1u << stage;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(S.a[stage]), sb = smem_u32(S.b[stage]);
                        const uint64_t ad = kAMN ? sdesc_mn_sw128(sa) : sdesc_sw128(sa);
                        const uint64_t bd = kBMN ? sdesc_mn_sw128(sb) : sdesc_sw128(sb);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (OP != GG_DW || kk < steps)
                                umma_pair<kF8>(d, ad + kk * a_step, bd + kk * b_step, idesc,
                                               ((!kF8 && kb > kb0) || kk > 0) ? 1u : 0u);
                        if (kF8) d += (uint32_t)ti.neff;
                        // GG_FP8_ROWS: one commit per block; the epilogue, which it wakes, frees the stage
                        if (!kRowsM) commit_pair(&S.empty[stage], 3u << lead);
                        if (++stage == kGgStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    commit_pair(&S.cfull[buf], 3u << lead);
                    if (++buf == 2) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
            umma_commit_pair_self(&S.done);
            drain_wait(&S.done, 0);
        } else if (warp >= 2 && kF8) {
            // -------------------------------------------- scale products
            const int tid = threadIdx.x - 64;
            const int kblocks = ceil_div(P.cdim, 128), fblocks = ceil_div(P.feat, 128);
            const bool wide = (kblocks & 3) == 0;  // rows of scales are 16-byte aligned
            int buf = 0, e = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e, part, splits);
                // GG_FP8: this CTA's features are one weight block, entry c is row c of the tile.
                // GG_FP8_ROWS: entry 128 h + r is this CTA's row r and weight block h of two.
                const int fb = ti.feat0 / 128 + (kRowsM ? 0 : (int)rank);
                const float* sw = P.a_scale + (long long)ti.e * fblocks * kblocks;
                for (int kb0 = 0; kb0 < ti.nkb; kb0 += kScaleBatch) {
                    // all loads of the batch in flight at once, and under the wait
                    constexpr int kW = kRowsM ? 2 : 1, kR = kRowsM ? 2 : kGgBN / 64;
                    float4 w[kW], v[kR];
#pragma unroll
                    for (int i = 0; i < kW; ++i)
                        w[i] = load_scales(sw + (long long)min(fb + i, fblocks - 1) * kblocks + ti.kb0 + kb0, kblocks - ti.kb0 - kb0, wide);
#pragma unroll
                    for (int i = 0; i < kR; ++i) {
                        const int c = tid + 64 * i, row = kRowsM ? (int)rank * 128 + c : c;
                        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (row < ti.ncols)
                            v[i] = load_scales(P.b_scale + (long long)(ti.row0 + row) * kblocks + ti.kb0 + kb0, kblocks - ti.kb0 - kb0,
                                               wide);
                    }
                    if (!wait_warp(&S.sempty[buf], bphase ^ 1u, S, P)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < kR; ++i) {
                        const int c = tid + 64 * i;
                        if (kRowsM) {  // an entry's four blocks side by side: its thread reads them at once
#pragma unroll
                            for (int j = 0; j < kW; ++j)
                                *reinterpret_cast<float4*>(&S.scale[buf][0][0] + 4 * (c + 128 * j)) =
                                    make_float4(v[i].x * w[j].x, v[i].y * w[j].y, v[i].z * w[j].z, v[i].w * w[j].w);
                        } else if (c < ti.neff) {
#pragma unroll
                            for (int j = 0; j < kW; ++j) {
                                S.scale[buf][0][c + 128 * j] = v[i].x * w[j].x;
                                S.scale[buf][1][c + 128 * j] = v[i].y * w[j].y;
                                S.scale[buf][2][c + 128 * j] = v[i].z * w[j].z;
                                S.scale[buf][3][c + 128 * j] = v[i].w * w[j].w;
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.sfull[buf]);
                    if (++buf == 2) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
        } else if (warp >= 2 && OP == GG_DW) {
            // -------------------------------------------- partial k-blocks
            const int tid = threadIdx.x - 64;
            int stage = 0, e = 0;
            uint32_t lphase = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e, part, splits);
                if (ti.nkb == 0) continue;
                stage = (stage + ti.nkb - 1) % kGgStages;  // of the tile's last k-block
                if (ti.rem) {
                    if (!wait_warp(&S.landed[stage], (lphase >> stage) & 1u, S, P)) {
                        ok = false;
                        break;
                    }
                    lphase ^= 1u << stage;
                    zero_rows(S.a[stage], 2, ti.rem, tid);
                    zero_rows(S.b[stage], ti.neff > 128 ? 2 : 1, ti.rem, tid);
                    fence_proxy_async_smem();
                    __syncwarp();
                    // the leader's MMAs read the zeros of both CTAs: the other one's have to be
                    // released at cluster scope, to the issuer's wait of the same scope
                    if (lane == 0) {
                        if (leader) mbar_arrive(&S.tail[stage]);
                        else mbar_arrive_cluster(mapa_shared(&S.tail[stage], lead));
                    }
                }
                if (++stage == kGgStages) stage = 0;
            }
        }
        if (kSplit && pair < ntiles) {  // the epilogue's exchange of partial sums
            __syncwarp();
            cluster_sync_all();
            cluster_sync_all();
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(GgRegs<OP>::kEpi));
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t cempty0 = mapa_shared(&S.cempty[0], lead);
        if (kRowsM) {
            epilogue_rows(P, S, pair, npairs, ntiles, rank, q, h, lane, tmem_base, cempty0);
        } else {
        int buf = 0, sbuf = 0, e = 0;
        uint32_t bphase = 0, sphase = 0;
        bool ok = true;
        for (int t = pair; t < ntiles && ok; t += npairs) {
            const GgTile ti = decode<OP>(P, S, t, e, part, splits);
            const int hc = ti.neff / 2, c0 = h * hc;  // this warp's accumulator columns c0 .. c0 + hc
            Acc acc;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[0][i][0] = acc[0][i][1] = acc[1][i][0] = acc[1][i][1] = 0ull;
            const int ck = kF8 ? blocks_per_drain(ti.neff) : P.chunk_kb;
            const int ng = (hc + 31) >> 5;  // 32-column groups; an odd 16 reads 16 columns that are not stored
            for (int kb0 = 0; kb0 < ti.nkb; kb0 += ck) {
                if (kF8 && kb0 % kScaleBatch == 0 && !wait_warp(&S.sfull[sbuf], sphase, S, P)) {
                    ok = false;
                    break;
                }
                if (!wait_warp(&S.cfull[buf], bphase, S, P)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kGgBN + c0);
                const float* sc = &S.scale[sbuf][kb0 % kScaleBatch][c0 + 2 * (lane & 3)];
                const int parts = kF8 ? min(ck, ti.nkb - kb0) : 1;
                const uint32_t release = cempty0 + 8u * (uint32_t)buf;
                for (int part = 0; part < parts; ++part) {
                    const bool last = part == parts - 1;
                    switch (ng) {
                        case 4: drain_columns<4, kF8>(acc, taddr, sc, last, release, lane); break;
                        case 3: drain_columns<3, kF8>(acc, taddr, sc, last, release, lane); break;
                        case 2: drain_columns<2, kF8>(acc, taddr, sc, last, release, lane); break;
                        default: drain_columns<1, kF8>(acc, taddr, sc, last, release, lane);
                    }
                    if (kF8) {
                        taddr += (uint32_t)ti.neff;
                        sc += kGgBN;
                    }
                }
                if (++buf == 2) {
                    buf = 0;
                    bphase ^= 1u;
                }
                if (kF8 && ((kb0 + ck) % kScaleBatch == 0 || kb0 + ck >= ti.nkb)) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.sempty[sbuf]);
                    if (++sbuf == 2) {
                        sbuf = 0;
                        sphase ^= 1u;
                    }
                }
            }
            if (kSplit) {
                cluster_sync_all();  // every pair's operands are read, so the first pair's stages are free
                if (ok && part > 0) send_partial(acc, S.a[0], part, rank, hc);
                cluster_sync_all();
                if (ok && part == 0) add_partials(acc, S.a[0], splits, hc);
            }
            if (!ok || part > 0) break;
            const int f = ti.feat0 + (int)rank * 128 + q * 32;
            const int nv = min(hc, ti.ncols - c0);
            const long long first = OP == GG_DW ? (long long)ti.e * P.cols + ti.col0 + c0 : (long long)ti.row0 + c0;
            if (f < P.feat)
                store_rows(acc, S.stage[warp - 4], static_cast<char*>(P.out) + (first * P.ldo + f) * (P.out_f32 ? 4 : 2),
                           P.ldo, nv, P.feat - f, P.out_f32, lane);
        }
        }
    }
    __syncthreads();
    tc_fence_before();
    cluster_sync_all();  // both CTAs done with TMEM and shared memory; the leader's MMAs have completed
    tc_fence_after();
    if (gave_up(S)) {  // the same in all CTAs of the cluster: nobody gives up after the barrier
        if (leader && threadIdx.x == 0) drain_loads(S, crank ^ 1u);
        __syncthreads();
        cluster_sync_all();
    }
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// Sets the kernel's shared memory once per device and checks the register
// split: setmaxnreg.inc would wait for ever if the launch brought fewer
// registers than kLaunchRegs per thread.
template <int OP, bool kSplit>
cudaError_t launch_op(const GgParams& P, int clusters, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;  // 0: set up at every launch
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, k_grouped<OP, kSplit>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(k_grouped<OP, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGgSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(k_grouped<OP, kSplit>, dim3(2 * P.splits * clusters), kGgThreads, kGgSmem, 2 * P.splits, s, P);
}

}  // namespace

cudaError_t launch_grouped(int op, const GgParams& params, cudaStream_t s) {
    GgParams P = params;
    // tiles, as an upper bound: the counts are on the device
    const long long ft = (P.feat + 255) / 256;
    const int groups = P.n_groups < P.n_rows ? P.n_groups : P.n_rows;
    const long long tiles = op == GG_DW ? ft * P.n_groups * ((P.cols + kGgBN - 1) / kGgBN)
                            : P.counts ? ft * (P.n_rows / kGgBN + groups + (P.zero_tail ? 1 : 0))
                                       : ft * ((P.n_rows + kGgBN - 1) / kGgBN);
    const int pairs = tc_num_sms() / 2;
    // Few tiles and a long contraction (32 k-blocks or more): the pairs of a cluster share it. Four
    // pairs where the exchange has room (128 rows) and all clusters of eight SMs run at once (about
    // a dozen do), else two. One group of 32 rows, 1024 x 8192: 32.8 -> 17.3 us (8-bit 25.3 -> 16.0);
    // eight groups of 4, 512 x 4096: 20.5 -> 16.5. At 16 k-blocks it costs more than it gains (8192 x
    // 1024, 100 rows: 12.3 against 14.5). 8-bit rows on M past 128 rows gain nothing and stay.
    P.splits = 1;
    if (op != GG_DW && P.cdim > 31 * (op < GG_FP8 ? 64 : 128)) {
        if (tiles <= 8 && P.n_rows <= 128) {
            P.splits = 4;
            if (op == GG_FP8_ROWS) op = GG_FP8;
        } else if (tiles <= 32 && op != GG_FP8_ROWS) {
            P.splits = 2;
        }
    }
    long long clusters = pairs;
    if (tiles < clusters || P.splits > 1) clusters = tiles;
    if (clusters < 1) return cudaSuccess;
    switch (op) {
        case GG_FWD: return P.splits > 1 ? launch_op<GG_FWD, true>(P, (int)clusters, s) : launch_op<GG_FWD, false>(P, (int)clusters, s);
        case GG_DX: return P.splits > 1 ? launch_op<GG_DX, true>(P, (int)clusters, s) : launch_op<GG_DX, false>(P, (int)clusters, s);
        case GG_FP8: return P.splits > 1 ? launch_op<GG_FP8, true>(P, (int)clusters, s) : launch_op<GG_FP8, false>(P, (int)clusters, s);
        case GG_DW: return launch_op<GG_DW, false>(P, (int)clusters, s);
        case GG_FP8_ROWS: return launch_op<GG_FP8_ROWS, false>(P, (int)clusters, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace lmoe
