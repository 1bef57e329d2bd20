// few.cu -- grouped products for a handful of rows (single tokens), bf16 and
// block-scaled 8-bit:
//
//     y[r, f] = sum_k x[r, k] W[e(r)][f, k]            (8-bit: each 128-block's sum times sx sw)
//
// Bound by reading each hit expert's weights once. The tcgen05 engine gives a
// 256-feature tile to a pair of SMs and keeps the tile's whole contraction there:
// a 1024 x 8192 matrix is 4 tiles, for 74 pairs. Here a CTA takes 16 features, its
// warps (eight or four) share the contraction and add up in shared memory, so every
// SM streams (24 warps, 16-byte loads, the next steps' in flight under this one's
// products). Device time by events (about 4 us of it the events'), one row, 8-bit
// weights: 2560 x 2048 8.2 us against 14.3, 1024 x 8192 14.3 against 26.6, 10240 x
// 8192 26.6 against 28.7; with 16 rows of one matrix the engine is as fast, with more
// it is faster, so up to 8 rows come here. Back to back (launches overlapping) those
// three take 3.8, 5.8 and 18.3 us (4.6 TB/s; a launch's start and end are 4 us of it).
// Measured no better: three to five steps ahead, the activations through the ring too (eight
// rows 29 us against 21), and CTAs that start at different places of the contraction.
//
// The multiplications are warp-level MMAs (m16n8, 16 features x 8 rows), which
// cost next to nothing beside the weight stream; on plain FMAs eight rows would
// take 9.5 instructions per weight. The order of the contraction inside an MMA is
// free as long as both operands share it, so a lane's 16 contiguous bytes of a
// weight row are the A fragments of two MMAs as they come, and the same 16 bytes
// of an activation row are their B fragments.
#include <cuda_bf16.h>

#include <atomic>

#include "grouped.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

constexpr int kFewFeats = 16;
constexpr int kFewSmWarps = 24;  // resident per SM: 80 registers a thread
static_assert(kFewRows <= 8, "one MMA's columns hold all rows");

struct FewParams {
    const uint8_t* w;       // [n_groups, feat, cdim]
    const uint8_t* x;       // [n_rows, cdim], row pitch ldx bytes
    long long ldx;
    const int* counts;      // null: one group of n_rows rows
    const float* w_scale;   // 8-bit: [n_groups, ceil(feat / 128), ceil(cdim / 128)]
    const float* x_scale;   // 8-bit: [n_rows, ceil(cdim / 128)]
    void* out;
    long long ldo;
    int n_groups, n_rows, slots, feat, cdim, out_f32;
};

template <bool kF8>
__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if (kF8)
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
            "%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Inclusive sum over the CTA's threads in thread order.
__device__ __forceinline__ int few_scan(int v, int* wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += wsum[w];
    return v;
}

// The slot-th group that has rows: {group, first row, rows}, or the rows behind
// the last group as {n_groups, first, rows} for slot = P.slots; no rows if there
// is none. Counts as in the engine: negative ones are 0, rows past n_rows do not
// exist.
template <int kWarps>
__device__ __forceinline__ int3 find_group(const FewParams& P, int slot, int* wsum, int* found) {
    constexpr int kPer = kMaxE / (32 * kWarps);
    if (threadIdx.x < 3) found[threadIdx.x] = 0;
    int c[kPer], rows = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = (int)threadIdx.x * kPer + i;
        c[i] = g < P.n_groups ? min(max(ld_global_s32(P.counts + g), 0), P.n_rows) : 0;
        rows += c[i];
    }
    const int end = few_scan(rows, wsum);  // at most 1024 x n_rows
    int at = end - rows, hit = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int lo = min(at, P.n_rows);
        at += c[i];
        c[i] = min(at, P.n_rows) - lo;
        hit += c[i] > 0;
    }
    int before = few_scan(hit, wsum) - hit;
    at = end - rows;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (c[i] > 0 && before++ == slot) {
            found[0] = (int)threadIdx.x * kPer + i;
            found[1] = min(at, P.n_rows);
            found[2] = c[i];
        }
        at += c[i];
    }
    if (slot == P.slots && threadIdx.x == 32 * kWarps - 1) {
        const int total = min(end, P.n_rows);
        found[0] = P.n_groups;
        found[1] = total;
        found[2] = P.n_rows - total;
    }
    __syncthreads();
    return make_int3(found[0], found[1], found[2]);
}

// 16 bytes to shared memory, asynchronously; zeros where there is nothing to read.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool in) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// The weights of a warp step (128 bytes of 16 rows) are four 16-byte pieces per thread. They
// come straight into registers, one step ahead, or (kRing) through shared memory, two
// steps ahead: [stage][piece][thread], each copied and read by its thread alone.
constexpr int kFewPieces = 4;

template <bool kF8, int kWarps, bool kRing>
__global__ void __launch_bounds__(32 * kWarps, kFewSmWarps / kWarps) k_few(const FewParams P) {
    constexpr int kStep = kF8 ? 128 : 64;  // contraction elements per step
    __shared__ float red[kWarps][kFewFeats][9];
    __shared__ int wsum[kWarps], found[3];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int3 grp = make_int3(0, 0, P.n_rows);
    dependent_wait_and_release();
    if (P.counts) grp = find_group<kWarps>(P, blockIdx.y, wsum, found);
    if (grp.z <= 0) return;
    const int f0 = blockIdx.x * kFewFeats;
    const long long row_bytes = (long long)P.cdim * (kF8 ? 1 : 2);
    const bool real = grp.x < P.n_groups;  // else zeros
    const int steps = real ? (P.cdim + kStep - 1) / kStep : 0;
    const int e = real ? grp.x : 0;
    // the lane's two weight rows, w8 bytes apart (past the end the first one again: its results are not stored)
    const uint8_t* w0 = P.w + ((long long)e * P.feat + f0 + g) * row_bytes + t * 16;
    const long long w8 = f0 + 8 < P.feat ? 8 * row_bytes : 0;
    const float* ws = kF8 ? P.w_scale + ((long long)e * ((P.feat + 127) / 128) + f0 / 128) * steps : nullptr;

    const bool has = g < grp.z;  // the lane's activation row
    const uint8_t* xr = P.x + (long long)(grp.y + (has ? g : 0)) * P.ldx + t * 16;
    const int c = 2 * t;       // the lane's output rows: columns 2 t and 2 t + 1 of the MMA
    const float* xs = kF8 ? P.x_scale + (long long)(grp.y + min(c, grp.z - 1)) * steps : nullptr;
    const int xs1 = c + 1 < grp.z ? steps : 0;
    extern __shared__ uint4 ring[];
    constexpr int kThreads = 32 * kWarps;
    const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
    uint4 na[kFewPieces], nb[2];
    auto fetch = [&](int s, int stage) {  // step s's weights
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const long long at = (long long)s * 128;
        const bool in0 = s < steps && at + t * 16 < row_bytes, in1 = s < steps && at + 64 + t * 16 < row_bytes;
        if (kRing) {
            const uint8_t* p0 = w0 + (in0 ? at : 0);
            const uint8_t* p1 = w0 + (in1 ? at + 64 : 0);
            const uint32_t to = mine + (uint32_t)(stage * kFewPieces * kThreads * 16);
            copy16(to, p0, in0);
            copy16(to + kThreads * 16, p0 + w8, in0);
            copy16(to + 2 * kThreads * 16, p1, in1);
            copy16(to + 3 * kThreads * 16, p1 + w8, in1);
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
            na[0] = in0 ? ld_global_v4(w0 + at) : zero;
            na[1] = in0 ? ld_global_v4(w0 + at + w8) : zero;
            na[2] = in1 ? ld_global_v4(w0 + at + 64) : zero;
            na[3] = in1 ? ld_global_v4(w0 + at + w8 + 64) : zero;
        }
    };
    float n0 = 0.f, n1 = 0.f;
    auto load = [&](int s) {  // and its activations and scales
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const long long at = (long long)s * 128;
        const bool in0 = s < steps && at + t * 16 < row_bytes, in1 = s < steps && at + 64 + t * 16 < row_bytes;
        nb[0] = in0 && has ? ld_global_v4(xr + at) : zero;
        nb[1] = in1 && has ? ld_global_v4(xr + at + 64) : zero;
        if (kF8 && s < steps) {
            const float sw = ld_global_f32(ws + s);
            n0 = ld_global_f32(xs + s) * sw;
            n1 = ld_global_f32(xs + xs1 + s) * sw;
        }
    };
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    // The lane's sums so far go to its own places in shared memory every 64 steps (4096 products):
    // the MMA's additions err towards zero, an fp32 result of 2^22 like-signed products came out
    // 0.3% low. 8-bit sums are drained every step, by the multiply-adds.
    float(&r0)[9] = red[warp][g], (&r1)[9] = red[warp][g + 8];
    auto drain = [&](bool first) {
        r0[c] = first ? acc[0] : r0[c] + acc[0];
        r0[c + 1] = first ? acc[1] : r0[c + 1] + acc[1];
        r1[c] = first ? acc[2] : r1[c] + acc[2];
        r1[c + 1] = first ? acc[3] : r1[c + 1] + acc[3];
    };
    constexpr int kDrain = 64;
    fetch(warp, 0);
    if (kRing) fetch(warp + kWarps, 1);
    load(warp);
    int stage = 0;
    for (int s = warp; s < steps; s += kWarps) {
        uint4 a[kFewPieces];
        const uint4 b[2] = {nb[0], nb[1]};
        const float s0 = n0, s1 = n1;
#pragma unroll
        for (int i = 0; i < kFewPieces; ++i) a[i] = na[i];
        if (s + kWarps < steps) {
            if (!kRing) fetch(s + kWarps, 0);
            load(s + kWarps);
        }
        if (kRing) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
            for (int i = 0; i < kFewPieces; ++i) a[i] = ring[(stage * kFewPieces + i) * kThreads + threadIdx.x];
        }
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        float(&o)[4] = kF8 ? d : acc;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mma_16x8<kF8>(o, a[2 * h].x, a[2 * h + 1].x, a[2 * h].y, a[2 * h + 1].y, b[h].x, b[h].y);
            mma_16x8<kF8>(o, a[2 * h].z, a[2 * h + 1].z, a[2 * h].w, a[2 * h + 1].w, b[h].z, b[h].w);
        }
        if (kF8) {
            acc[0] = fmaf(d[0], s0, acc[0]);
            acc[1] = fmaf(d[1], s1, acc[1]);
            acc[2] = fmaf(d[2], s0, acc[2]);
            acc[3] = fmaf(d[3], s1, acc[3]);
        }
        if (kRing) {
            fetch(s + 2 * kWarps, stage);
            stage ^= 1;
        }
        if (!kF8 && s / kWarps % kDrain == kDrain - 1) {
            drain(s / kWarps < kDrain);
            acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
        }
    }
    if (kRing) asm volatile("cp.async.wait_all;" ::: "memory");
    drain(kF8 || steps <= warp + kWarps * (kDrain - 1));
    __syncthreads();
    static_assert(32 * kWarps >= kFewFeats * 8, "a thread per output");
    if (threadIdx.x < kFewFeats * 8) {
        const int f = threadIdx.x % kFewFeats, r = threadIdx.x / kFewFeats;
        if (f0 + f < P.feat && r < grp.z) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) v += red[q][f][r];
            const long long o = (long long)(grp.y + r) * P.ldo + f0 + f;
            if (P.out_f32) static_cast<float*>(P.out)[o] = v;
            else static_cast<__nv_bfloat16*>(P.out)[o] = __float2bfloat16_rn(v);
        }
    }
}

// A grid of four-warp CTAs that fits at once. It is given as much shared memory per CTA as
// leaves room for ceil(grid / SMs) of them: with more room the next launch's CTAs, which
// may come in early, would settle unevenly in the gaps, and that launch then wait for the
// fullest SM.
template <bool kF8>
cudaError_t launch_ring(const FewParams& P, dim3 grid, int per_sm, cudaStream_t s) {
    constexpr int kSmShared = 228 * 1024, kWarps = 4;
    constexpr int kFixed = (int)sizeof(float) * kWarps * kFewFeats * 9 + 64 + 1024;  // static, and the system's
    static_assert(kSmShared / (kFewSmWarps / kWarps) - kFixed - 640 >= 2 * kFewPieces * 32 * kWarps * 16, "the ring's room");
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(k_few<kF8, kWarps, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmShared / (kFewSmWarps / 8 + 1));  // per_sm is above kFewSmWarps / 8
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    const int room = (kSmShared / per_sm - kFixed - 512) & ~127;
    return launch_dependent(k_few<kF8, kWarps, true>, grid, 32 * kWarps, room, 0, s, P);
}

}  // namespace

cudaError_t launch_few(bool f8, const void* w, const void* x, long long ldx_bytes, const GgParams& G, cudaStream_t s) {
    FewParams P;
    P.w = static_cast<const uint8_t*>(w);
    P.x = static_cast<const uint8_t*>(x);
    P.ldx = ldx_bytes;
    P.counts = G.counts;
    P.w_scale = G.a_scale;
    P.x_scale = G.b_scale;
    P.out = G.out;
    P.ldo = G.ldo;
    P.n_groups = G.n_groups;
    P.n_rows = G.n_rows;
    P.slots = G.counts ? (G.n_rows < G.n_groups ? G.n_rows : G.n_groups) : 1;
    P.feat = G.feat;
    P.cdim = G.cdim;
    P.out_f32 = G.out_f32;
    const dim3 grid((G.feat + kFewFeats - 1) / kFewFeats, P.slots + (G.counts && G.zero_tail ? 1 : 0));
    // Eight warps per CTA where all those CTAs fit at once: its contraction is shared by more (1024 x 8192, one
    // row: 5.8 us; four warps 8.7, the ring 7.2). Beyond that four, as twice as many CTAs are resident: through
    // the ring, two steps ahead, while they fit at once (10240 x 8192, 8-bit: 18.3 us, registers 20.8, eight
    // warps 21.8; 8192 x 8192 bf16 25.3, 33.2, 32.6), else through registers (8 rows in 8 of 64 groups, 5120 x
    // 2048, 8-bit: 22.0, ring 23.1, eight warps 28.4).
    const long long ctas = (long long)grid.x * grid.y, per_sm = (ctas + tc_num_sms() - 1) / tc_num_sms();
    if (per_sm <= kFewSmWarps / 8)
        return f8 ? launch_dependent(k_few<true, 8, false>, grid, 256, 0, 0, s, P)
                  : launch_dependent(k_few<false, 8, false>, grid, 256, 0, 0, s, P);
    if (per_sm <= kFewSmWarps / 4)
        return f8 ? launch_ring<true>(P, grid, (int)per_sm, s) : launch_ring<false>(P, grid, (int)per_sm, s);
    return f8 ? launch_dependent(k_few<true, 4, false>, grid, 128, 0, 0, s, P)
              : launch_dependent(k_few<false, 4, false>, grid, 128, 0, 0, s, P);
}

}  // namespace lmoe
