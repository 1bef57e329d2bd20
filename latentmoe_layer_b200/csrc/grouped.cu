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
//
// Why the features are on M. A batch's groups are uneven, and rows on M would
// be padded to 256 per group; the MMA's N takes any multiple of 32, so the
// ragged end of a group costs its own rows only, and a decode batch (a few rows
// per expert) streams each weight tile once with N = 32. It also makes lanes
// consecutive in the output's fast axis, so stores need no transposition.
//
// Why pairs. 128 x 256 tiles on single SMs read 48 KB of operands per 64-deep
// k-block, 96 bytes per SM and cycle at the tensor peak; a pair's 256 x 256 tile
// (tcgen05.mma.cta_group::2) reads 32 KB per SM for the same work.
//
// Structure of one CTA of a pair (one pair per two SMs, persistent over tiles):
//   warp 0       TMA producer (own 128 features of A, own half of B's rows)
//   warp 1       TMEM owner; in the leader CTA, lane 0 issues the MMAs
//   warps 2, 3   GG_FP8: the products sx * sw of the next four k-blocks, into
//                shared memory; GG_DW: a group's last, partial k-block
//   warps 4-11   epilogue: drain TMEM chunks into fp32 registers, store
// Tiles are found from prefix sums of the counts that every CTA builds in
// shared memory, so a call is one launch and needs no workspace.
//
// Accumulation: TMEM holds a chunk of the contraction (two buffers of 256
// columns), the epilogue adds chunks into fp32 registers while the next one
// runs. GG_FP8 drains every 128-deep block, where its two scales are applied
// as one fused multiply-add per element (their product is rounded to fp32
// once). fp32 outputs drain every 512, which keeps the tensor core's
// accumulation error near that of fp32 additions; bf16 outputs, whose rounding
// is three orders larger, accumulate the whole contraction in TMEM.
//
// A group's rows that do not fill a k-block of GG_DW (the contraction runs over
// rows) must not meet the next group's, which may hold anything: warps 2 and 3
// copy that k-block with plain loads and write zeros behind the last row.
// Elsewhere rows of a neighbouring group land in output rows that are not
// stored. Features and contraction indices past the matrix are zero-filled by
// the tensor maps.
//
// Every mbarrier wait is bounded; on running out the kernel records
// LMOE_ERR_TIMEOUT, drains its own MMAs, frees TMEM and returns.
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
// registers per thread: 128 x kProdRegs + 256 x kEpiRegs must not exceed 384 x kLaunchRegs
constexpr int kLaunchRegs = 168, kProdRegs = 56, kEpiRegs = 224;
static_assert(128 * kProdRegs + 256 * kEpiRegs <= 384 * kLaunchRegs, "register split");

struct alignas(1024) GgShared {
    uint8_t a[kGgStages][kGgABytes];
    uint8_t b[kGgStages][kGgBBytes];
    float scale[2][kScaleBatch][kGgBN];
    int off[kMaxE + 2];    // first row of each group, then the end of the last group, then n_rows
    int tiles[kMaxE + 2];  // tile prefix per group
    long long wsum[kGgThreads / 32];
    uint64_t full[kGgStages], empty[kGgStages];
    uint64_t tailreq[kGgStages], tail[kGgStages];  // GG_DW: stage handed to the copying warps, and back
    uint64_t cfull[2], cempty[2], sfull[2], sempty[2], done;
    uint32_t tmem;
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
        mine += P.counts ? min(max(__ldg(P.counts + g), 0), P.n_rows) : P.n_rows;
    long long end = block_scan(mine, S.wsum);
    long long at = end - mine;
    long long mt = 0;
    for (int g = g0; g < g1; ++g) {
        const int c = P.counts ? min(max(__ldg(P.counts + g), 0), P.n_rows) : P.n_rows;
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
        const int c = P.counts ? min(max(__ldg(P.counts + g), 0), P.n_rows) : P.n_rows;
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
    int nkb;    // k-blocks
    int rem;    // GG_DW: rows of the last k-block when it is partial, else 0
};

// Tile t. Within a group, raster blocks of kGgRaster N-side tiles sweep the
// features, so that the pairs running at once share both operands in L2.
// `e` carries the last tile's group: a CTA's tiles only move forward.
template <int OP>
__device__ __forceinline__ GgTile decode(const GgParams& P, const GgShared& S, int t, int& e) {
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
    GgTile ti;
    ti.e = e;
    ti.feat0 = (r / ms) * 256;
    if (OP == GG_DW) {
        ti.row0 = S.off[e];
        ti.col0 = c * kGgBN;
        ti.ncols = min(kGgBN, P.cols - ti.col0);
        ti.nkb = ceil_div(cnt, 64);
        ti.rem = cnt & 63;
    } else {
        ti.row0 = S.off[e] + c * kGgBN;
        ti.col0 = 0;
        ti.ncols = min(kGgBN, cnt - c * kGgBN);
        ti.nkb = e < P.n_groups ? ceil_div(P.cdim, OP == GG_FP8 ? 128 : 64) : 0;
        ti.rem = 0;
    }
    ti.neff = (ti.ncols + 31) & ~31;
    return ti;
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t leader_bar, int x, int y,
                                                 int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

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

// try_wait that acquires at cluster scope: the arrivals come from both CTAs.
__device__ __forceinline__ bool mbar_wait_bounded_cluster(uint64_t* bar, uint32_t parity, unsigned limit, int* err) {
    for (unsigned i = 0; i < limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 4095u) == 4095u && *(volatile int*)err != 0) return false;
    }
    atomicCAS(err, 0, 5);
    return false;
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// GG_DW: 64 threads copy the last, partial k-block of one operand: 64
// contraction rows (rows row .. row + rem of src, zeros behind) x `width`
// columns from column c0, zeros past column `limit`. Sub-tiles of 64 columns,
// 128-byte rows, 16-byte pieces swizzled by the row's index modulo 8.
__device__ __forceinline__ void copy_partial(uint8_t* dst, const uint16_t* src, long long ld, int row, int rem, int c0,
                                             int limit, int width, int tid) {
    const int pieces = width / 8;  // 16-byte pieces per row, a multiple of 8
    for (int i0 = tid; i0 < 64 * pieces; i0 += 64 * 4) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 64 * u;
            const int r = i / pieces, c = c0 + (i % pieces) * 8;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rem && c < limit)
                v[u] = __ldg(reinterpret_cast<const uint4*>(src + (long long)(row + r) * ld + c));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 64 * u;
            const int r = i / pieces, q = i % pieces;
            if (r < 64)
                *reinterpret_cast<uint4*>(dst + (q >> 3) * 8192 + r * 128 + (((q & 7) ^ (r & 7)) << 4)) = v[u];
        }
    }
}

template <int OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGgThreads, 1) k_grouped(const __grid_constant__ GgParams P) {
    constexpr bool kF8 = OP == GG_FP8, kAMN = OP == GG_DX || OP == GG_DW, kBMN = OP == GG_DW;
    extern __shared__ uint8_t smem_raw[];
    GgShared& S = *reinterpret_cast<GgShared*>(smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw)));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kGgStages; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
            mbar_init(&S.tailreq[s], 1);
            mbar_init(&S.tail[s], 4);  // two copying warps in each CTA
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.cfull[b], 1);
            mbar_init(&S.cempty[b], 2 * kGgEpiWarps);  // both CTAs' epilogue warps
            mbar_init(&S.sfull[b], 2);
            mbar_init(&S.sempty[b], kGgEpiWarps);
        }
        mbar_init(&S.done, 1);
        fence_mbar_init();
        prefetch_tmap(&P.a_map);
        prefetch_tmap(&P.b_map);
        if (!kBMN) prefetch_tmap(&P.b_small);
    }
    if (warp == 1) {
        tmem_alloc_pair(&S.tmem, 512);
        tmem_relinquish_pair();
    }
    const int ntiles = build_groups<OP>(P, S);
    tc_fence_before();
    cluster_sync_all();  // barriers, TMEM and tables of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem_base = S.tmem;
    int* err = P.err;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProdRegs));
        if (warp == 0 && lane == 0) {
            // -------------------------------------------- TMA producer (both CTAs)
            int stage = 0, e = 0;
            uint32_t phase = 0, issued = 0, issued_par = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e);
                const int half = ti.neff / 2, f0 = ti.feat0 + (int)rank * 128;
                const int b0 = (kBMN ? ti.col0 : ti.row0) + (int)rank * half;
                const uint32_t bytes_b = kBMN ? (uint32_t)((half + 63) / 64) * 8192u : (uint32_t)half * 128u;
                for (int kb = 0; kb < ti.nkb; ++kb) {
                    if (!mbar_wait_bounded(&S.empty[stage], phase ^ 1u, P.spin, err)) {
                        ok = false;
                        break;
                    }
                    if (OP == GG_DW && ti.rem && kb == ti.nkb - 1) {
                        // warps 2 and 3 fill this stage; its earlier load has been consumed
                        mbar_arrive(&S.tailreq[stage]);
                        if (leader) mbar_arrive(&S.full[stage]);
                        issued &= ~(1u << stage);
                    } else {
                        if (leader) mbar_arrive_expect_tx(&S.full[stage], 2u * (kGgABytes + bytes_b));
                        const uint32_t bar = mapa_shared(&S.full[stage], 0);
                        if (OP == GG_FWD || OP == GG_FP8) {
                            tma_load_3d_pair(S.a[stage], &P.a_map, bar, kb * (kF8 ? 128 : 64), f0, ti.e);
                        } else if (OP == GG_DX) {
                            tma_load_3d_pair(S.a[stage], &P.a_map, bar, f0, kb * 64, ti.e);
                            tma_load_3d_pair(S.a[stage] + 8192, &P.a_map, bar, f0 + 64, kb * 64, ti.e);
                        } else {
                            const int r = ti.row0 + kb * 64;
                            tma_load_3d_pair(S.a[stage], &P.a_map, bar, f0, r, 0);
                            tma_load_3d_pair(S.a[stage] + 8192, &P.a_map, bar, f0 + 64, r, 0);
                            tma_load_3d_pair(S.b[stage], &P.b_map, bar, b0, r, 0);
                            if (half > 64) tma_load_3d_pair(S.b[stage] + 8192, &P.b_map, bar, b0 + 64, r, 0);
                        }
                        if (!kBMN) {
                            const int x = kb * (kF8 ? 128 : 64);
                            if (half == 128) {
                                tma_load_3d_pair(S.b[stage], &P.b_map, bar, x, b0, 0);
                            } else {  // the ragged end: boxes of 16 rows
                                for (int r = 0; r < half; r += 16)
                                    tma_load_3d_pair(S.b[stage] + r * 128, &P.b_small, bar, x, b0 + r, 0);
                            }
                        }
                        issued |= 1u << stage;
                        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                    }
                    if (++stage == kGgStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the leader's full barriers count both CTAs' bytes: waiting on them drains every
            // load of the pair before either CTA can pass the final cluster barrier
            if (leader)
                for (int s = 0; s < kGgStages; ++s)
                    if ((issued >> s) & 1u) mbar_wait_bounded(&S.full[s], (issued_par >> s) & 1u, 1u << 26, err);
        } else if (warp == 1 && lane == 0 && leader) {
            // -------------------------------------------- MMA issuer (leader only)
            constexpr uint32_t type = kF8 ? 0u : 1u;  // e4m3 : bf16
            constexpr uint32_t idesc0 = (1u << 4) | (type << 7) | (type << 10) | ((kAMN ? 1u : 0u) << 15) |
                                        ((kBMN ? 1u : 0u) << 16) | ((256u >> 4) << 24);
            constexpr uint64_t a_step = kAMN ? 2048 >> 4 : 32 >> 4, b_step = kBMN ? 2048 >> 4 : 32 >> 4;
            int stage = 0, buf = 0, e = 0;
            uint32_t phase = 0, bphase = 0, tphase = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e);
                const uint32_t idesc = idesc0 | ((uint32_t)(ti.neff >> 3) << 17);
                const int ck = kF8 ? 1 : P.chunk_kb;
                for (int kb0 = 0; kb0 < ti.nkb && ok; kb0 += ck) {
                    if (!mbar_wait_bounded(&S.cempty[buf], bphase ^ 1u, P.spin, err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(buf * kGgBN);
                    const int kb1 = min(ti.nkb, kb0 + ck);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!mbar_wait_bounded(&S.full[stage], phase, P.spin, err)) {
                            ok = false;
                            break;
                        }
                        if (OP == GG_DW && ti.rem && kb == ti.nkb - 1) {
                            if (!mbar_wait_bounded_cluster(&S.tail[stage], (tphase >> stage) & 1u, P.spin, err)) {
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
                            umma_pair<kF8>(d, ad + kk * a_step, bd + kk * b_step, idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
                        umma_commit_pair_both(&S.empty[stage]);
                        if (++stage == kGgStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair_both(&S.cfull[buf]);
                    if (++buf == 2) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
            umma_commit_pair_self(&S.done);
            mbar_wait_bounded(&S.done, 0, 1u << 26, err);
        } else if (warp >= 2 && kF8) {
            // -------------------------------------------- scale products
            const int tid = threadIdx.x - 64;
            const int kblocks = ceil_div(P.cdim, 128), fblocks = ceil_div(P.feat, 128);
            const bool wide = (kblocks & 3) == 0;  // rows of scales are 16-byte aligned
            int buf = 0, e = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e);
                const int fb = ti.feat0 / 128 + (int)rank;
                const float* sw = P.a_scale + ((long long)ti.e * fblocks + min(fb, fblocks - 1)) * kblocks;
                for (int kb0 = 0; kb0 < ti.nkb; kb0 += kScaleBatch) {
                    if (!mbar_wait_bounded(&S.sempty[buf], bphase ^ 1u, P.spin, err)) {
                        ok = false;
                        break;
                    }
                    float w[kScaleBatch];
#pragma unroll
                    for (int q = 0; q < kScaleBatch; ++q) w[q] = kb0 + q < kblocks ? __ldg(sw + kb0 + q) : 0.f;
#pragma unroll
                    for (int i = 0; i < kGgBN / 64; ++i) {
                        const int c = tid + 64 * i;
                        if (c >= ti.neff) break;
                        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (c < ti.ncols) {
                            const float* p = P.b_scale + (long long)(ti.row0 + c) * kblocks + kb0;
                            if (wide) {
                                s = __ldg(reinterpret_cast<const float4*>(p));
                            } else {
                                s.x = __ldg(p);
                                if (kb0 + 1 < kblocks) s.y = __ldg(p + 1);
                                if (kb0 + 2 < kblocks) s.z = __ldg(p + 2);
                                if (kb0 + 3 < kblocks) s.w = __ldg(p + 3);
                            }
                        }
                        S.scale[buf][0][c] = s.x * w[0];
                        S.scale[buf][1][c] = s.y * w[1];
                        S.scale[buf][2][c] = s.z * w[2];
                        S.scale[buf][3][c] = s.w * w[3];
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
            // These warps may be many rounds of the ring ahead of the loads, so a stage's own
            // barriers say nothing to them: the producer hands the stage over.
            int stage = 0, e = 0;
            uint32_t rphase = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                const GgTile ti = decode<OP>(P, S, t, e);
                if (ti.nkb == 0) continue;
                stage = (stage + ti.nkb - 1) % kGgStages;  // of the tile's last k-block
                if (ti.rem) {
                    if (!mbar_wait_bounded(&S.tailreq[stage], (rphase >> stage) & 1u, P.spin, err)) {
                        ok = false;
                        break;
                    }
                    rphase ^= 1u << stage;
                    const int row = ti.row0 + (ti.nkb - 1) * 64, half = ti.neff / 2;
                    copy_partial(S.a[stage], P.x, P.ldx, row, ti.rem, ti.feat0 + (int)rank * 128, P.feat, 128, tid);
                    copy_partial(S.b[stage], P.dy, P.lddy, row, ti.rem, ti.col0 + (int)rank * half, P.cols,
                                 (half + 63) & ~63, tid);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(&S.tail[stage], 0));
                }
                if (++stage == kGgStages) stage = 0;
            }
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        const int q = warp & 3, h = (warp - 4) >> 2;
        int buf = 0, sbuf = 0, e = 0;
        uint32_t bphase = 0, sphase = 0;
        bool ok = true;
        for (int t = pair; t < ntiles && ok; t += npairs) {
            const GgTile ti = decode<OP>(P, S, t, e);
            const int hc = ti.neff / 2, c0 = h * hc;  // this warp's accumulator columns c0 .. c0 + hc
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
            const int ck = kF8 ? 1 : P.chunk_kb;
            for (int kb0 = 0; kb0 < ti.nkb; kb0 += ck) {
                if (kF8 && kb0 % kScaleBatch == 0 && !mbar_wait_bounded(&S.sfull[sbuf], sphase, P.spin, err)) {
                    ok = false;
                    break;
                }
                if (!mbar_wait_bounded(&S.cfull[buf], bphase, P.spin, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kGgBN + c0);
                const float* sc = &S.scale[sbuf][kb0 % kScaleBatch][c0];
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c < hc) {
                        uint32_t r0[16], r1[16];
                        tmem_ld16(taddr + (uint32_t)c, r0);
                        if (c + 16 < hc) tmem_ld16(taddr + (uint32_t)(c + 16), r1);
                        tmem_ld_wait();
                        if (kF8) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                const float4 s = *reinterpret_cast<const float4*>(sc + c + i);
                                uint64_t* a = &acc[(c + i) / 2];
                                a[0] = fma2(pack2(r0[i], r0[i + 1]), pack2(__float_as_uint(s.x), __float_as_uint(s.y)), a[0]);
                                a[1] = fma2(pack2(r0[i + 2], r0[i + 3]), pack2(__float_as_uint(s.z), __float_as_uint(s.w)), a[1]);
                            }
                            if (c + 16 < hc) {
#pragma unroll
                                for (int i = 0; i < 16; i += 4) {
                                    const float4 s = *reinterpret_cast<const float4*>(sc + c + 16 + i);
                                    uint64_t* a = &acc[(c + 16 + i) / 2];
                                    a[0] = fma2(pack2(r1[i], r1[i + 1]), pack2(__float_as_uint(s.x), __float_as_uint(s.y)), a[0]);
                                    a[1] = fma2(pack2(r1[i + 2], r1[i + 3]), pack2(__float_as_uint(s.z), __float_as_uint(s.w)), a[1]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                acc[c / 2 + i] = add2(acc[c / 2 + i], pack2(r0[2 * i], r0[2 * i + 1]));
                            if (c + 16 < hc) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    acc[c / 2 + 8 + i] = add2(acc[c / 2 + 8 + i], pack2(r1[2 * i], r1[2 * i + 1]));
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(&S.cempty[buf], 0));
                if (++buf == 2) {
                    buf = 0;
                    bphase ^= 1u;
                }
                if (kF8 && (kb0 % kScaleBatch == kScaleBatch - 1 || kb0 == ti.nkb - 1)) {
                    if (lane == 0) mbar_arrive(&S.sempty[sbuf]);
                    if (++sbuf == 2) {
                        sbuf = 0;
                        sphase ^= 1u;
                    }
                }
            }
            if (!ok) break;
            // lanes hold consecutive features: 64 (bf16) or 128 (fp32) contiguous bytes per row and warp
            const int f = ti.feat0 + (int)rank * 128 + q * 32 + lane;
            const int nv = f < P.feat ? min(hc, ti.ncols - c0) : 0;
            const long long first = OP == GG_DW ? (long long)ti.e * P.cols + ti.col0 + c0 : (long long)ti.row0 + c0;
            const long long at = first * P.ldo + f;
            if (P.out_f32) {
                float* o = static_cast<float*>(P.out) + at;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    float lo, hi;
                    unpack2(acc[i], lo, hi);
                    if (2 * i < nv) *o = lo;
                    o += P.ldo;
                    if (2 * i + 1 < nv) *o = hi;
                    o += P.ldo;
                }
            } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(P.out) + at;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    float lo, hi;
                    unpack2(acc[i], lo, hi);
                    if (2 * i < nv) *o = __float2bfloat16_rn(lo);
                    o += P.ldo;
                    if (2 * i + 1 < nv) *o = __float2bfloat16_rn(hi);
                    o += P.ldo;
                }
            }
        }
    }
    __syncthreads();
    tc_fence_before();
    cluster_sync_all();  // both CTAs done with TMEM and shared memory; the leader's MMAs have completed
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// Sets the kernel's shared memory once per device and checks the register
// split: setmaxnreg.inc would wait for ever if the launch brought fewer
// registers than kLaunchRegs per thread.
template <int OP>
cudaError_t launch_op(const GgParams& P, int pairs, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, k_grouped<OP>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(k_grouped<OP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGgSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    k_grouped<OP><<<2 * pairs, kGgThreads, kGgSmem, s>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped(int op, const GgParams& P, cudaStream_t s) {
    // no more pairs than tiles: an upper bound, the counts are on the device
    const long long ft = (P.feat + 255) / 256;
    const long long ct = op == GG_DW ? (long long)P.n_groups * ((P.cols + kGgBN - 1) / kGgBN)
                                     : (long long)P.n_rows / kGgBN + P.n_groups + (P.zero_tail ? 1 : 0);
    long long pairs = tc_num_sms() / 2;
    if (ft * ct < pairs) pairs = ft * ct;
    if (pairs < 1) return cudaSuccess;
    switch (op) {
        case GG_FWD: return launch_op<GG_FWD>(P, (int)pairs, s);
        case GG_DX: return launch_op<GG_DX>(P, (int)pairs, s);
        case GG_DW: return launch_op<GG_DW>(P, (int)pairs, s);
        case GG_FP8: return launch_op<GG_FP8>(P, (int)pairs, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace lmoe
