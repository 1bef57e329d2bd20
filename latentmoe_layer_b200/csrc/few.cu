// few.cu -- grouped products for a handful of rows (single tokens), bf16 and
// block-scaled 8-bit:
//
//     y[r, f] = sum_k x[r, k] W[e(r)][f, k]            (8-bit: each 128-block's sum times sx sw)
//
// Bound by reading each hit expert's weights once. The tcgen05 engine gives a
// 256-feature tile to a pair of SMs and keeps the tile's whole contraction there:
// a 1024 x 8192 matrix is 4 tiles, for 74 pairs. Here a CTA takes 16 features, its
// warps (eight or four) share the contraction and add up in shared memory, so every
// SM streams (24 warps, 16-byte loads, the next step's in flight under this one's
// products). Device time by events (about 4 us of it the events'), one row, 8-bit
// weights: 2560 x 2048 8.2 us against 14.3, 1024 x 8192 14.3 against 26.6, 10240 x
// 8192 26.6 against 28.7; with 16 rows of one matrix the engine is as fast, with more
// it is faster, so up to 8 rows come here. Back to back (launches overlapping) those
// three take 3.8, 5.9 and 21.3 us (4 TB/s: a launch's start and end cost 4 us of it).
// Deeper rings of asynchronous copies in shared memory measured the same for one row
// and worse for eight (29 us against 22: the activations are read again per CTA).
//
// The multiplications are warp-level MMAs (m16n8, 16 features x 8 rows), which
// cost next to nothing beside the weight stream; on plain FMAs eight rows would
// take 9.5 instructions per weight. The order of the contraction inside an MMA is
// free as long as both operands share it, so a lane's 16 contiguous bytes of a
// weight row are the A fragments of two MMAs as they come, and the same 16 bytes
// of an activation row are their B fragments.
#include <cuda_bf16.h>

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
    int n_groups, n_rows, slots, feat, cdim, out_f32, zero_tail;
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
        c[i] = g < P.n_groups ? min(max(__ldg(P.counts + g), 0), P.n_rows) : 0;
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

// One warp step's operands: 128 bytes of 16 weight rows and of 8 activation rows,
// and the 8-bit scales of the lane's two output rows.
struct Step {
    uint4 a[4], b[2];
    float s0, s1;
};

template <bool kF8, int kWarps>
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
    auto load = [&](int s, Step& v) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const long long at = (long long)s * 128;
        const bool in0 = s < steps && at + t * 16 < row_bytes, in1 = s < steps && at + 64 + t * 16 < row_bytes;
        v.a[0] = in0 ? ld_global_nc_v4(reinterpret_cast<const uint4*>(w0 + at)) : zero;
        v.a[1] = in0 ? ld_global_nc_v4(reinterpret_cast<const uint4*>(w0 + at + w8)) : zero;
        v.a[2] = in1 ? ld_global_nc_v4(reinterpret_cast<const uint4*>(w0 + at + 64)) : zero;
        v.a[3] = in1 ? ld_global_nc_v4(reinterpret_cast<const uint4*>(w0 + at + w8 + 64)) : zero;
        v.b[0] = in0 && has ? ld_global_nc_v4(reinterpret_cast<const uint4*>(xr + at)) : zero;
        v.b[1] = in1 && has ? ld_global_nc_v4(reinterpret_cast<const uint4*>(xr + at + 64)) : zero;
        if (kF8 && s < steps) {
            const float sw = __ldg(ws + s);
            v.s0 = __ldg(xs + s) * sw;
            v.s1 = __ldg(xs + xs1 + s) * sw;
        }
    };
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    Step v;
    load(warp, v);
    for (int s = warp; s < steps; s += kWarps) {
        const Step q = v;
        if (s + kWarps < steps) load(s + kWarps, v);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        float(&o)[4] = kF8 ? d : acc;
        mma_16x8<kF8>(o, q.a[0].x, q.a[1].x, q.a[0].y, q.a[1].y, q.b[0].x, q.b[0].y);
        mma_16x8<kF8>(o, q.a[0].z, q.a[1].z, q.a[0].w, q.a[1].w, q.b[0].z, q.b[0].w);
        mma_16x8<kF8>(o, q.a[2].x, q.a[3].x, q.a[2].y, q.a[3].y, q.b[1].x, q.b[1].y);
        mma_16x8<kF8>(o, q.a[2].z, q.a[3].z, q.a[2].w, q.a[3].w, q.b[1].z, q.b[1].w);
        if (kF8) {
            acc[0] = fmaf(d[0], q.s0, acc[0]);
            acc[1] = fmaf(d[1], q.s1, acc[1]);
            acc[2] = fmaf(d[2], q.s0, acc[2]);
            acc[3] = fmaf(d[3], q.s1, acc[3]);
        }
    }
    red[warp][g][2 * t] = acc[0];
    red[warp][g][2 * t + 1] = acc[1];
    red[warp][g + 8][2 * t] = acc[2];
    red[warp][g + 8][2 * t + 1] = acc[3];
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
    P.zero_tail = G.zero_tail;
    const dim3 grid((G.feat + kFewFeats - 1) / kFewFeats, P.slots + (G.counts && G.zero_tail ? 1 : 0));
    // Four warps per CTA where that still fills the SMs (more than a wave of eight-warp CTAs): twice as many
    // CTAs are resident, so the last wave wastes less (8 rows in 8 of 64 groups, 5120 x 2048, 8-bit 28.4 ->
    // 22.5 us; 128 groups of 2560 x 2048 15.3 -> 13.8; 10240 x 8192 21.8 -> 21.3). Eight where the grid is
    // small, so that a CTA's contraction is shared by more (1024 x 8192: 5.9 us against 8.7).
    if ((long long)grid.x * grid.y > (long long)tc_num_sms() * (kFewSmWarps / 8))
        return f8 ? launch_dependent(k_few<true, 4>, grid, 128, 0, 0, s, P)
                  : launch_dependent(k_few<false, 4>, grid, 128, 0, 0, s, P);
    return f8 ? launch_dependent(k_few<true, 8>, grid, 256, 0, 0, s, P)
              : launch_dependent(k_few<false, 8>, grid, 256, 0, 0, s, P);
}

}  // namespace lmoe
