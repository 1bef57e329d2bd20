// fp8.cu -- 8-bit quantisation with one fp32 scale per block of 128.
//
//   a = max(amax over the block, 2^-100)    scale = a / 448
//   code = nearest e4m3 to x * (448 / a), saturating at 448
//
// every step an fp32 operation rounded to nearest (__fdiv_rn, __fmul_rn), so
// the bytes do not depend on contraction or order. The floor 2^-100 keeps
// 448 / a finite: a zero block gets zero codes. The maximum is taken over the
// bit patterns of |x|, in which a NaN is above infinity: a NaN makes its block
// NaN, an infinity makes the block's scale infinite.
//
// Both kernels are bound by HBM (3 bytes per bf16 element): every element is
// read once into registers with 16-byte loads, its block's maximum is taken
// with warp shuffles, and its code is written from the same registers.
#include <cuda_fp8.h>

#include "grouped.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

// Eight elements as loaded: their values and the largest |x| pattern.
template <bool kF32>
struct Eight {
    uint4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ void zero() {
        w[0] = make_uint4(0u, 0u, 0u, 0u);
        if (kF32) w[kF32 ? 1 : 0] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void load(const void* p) {  // 16-byte aligned
        w[0] = ld_global_v4(static_cast<const uint4*>(p));
        if (kF32) w[kF32 ? 1 : 0] = ld_global_v4(static_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ uint32_t amax() const {
        if (kF32) {
            const uint32_t m = 0x7FFFFFFFu;
            const uint4 a = w[0], b = w[kF32 ? 1 : 0];
            return max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)), max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
        }
        const uint32_t m = 0x7FFF7FFFu;  // two bf16 patterns per word
        const uint32_t q = __vmaxu2(__vmaxu2(w[0].x & m, w[0].y & m), __vmaxu2(w[0].z & m, w[0].w & m));
        return max(q << 16, q & 0xFFFF0000u);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kF32) {
                v[i] = __uint_as_float(a[i]);
            } else {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
            }
        }
        if (kF32) {
            const uint4 b = w[kF32 ? 1 : 0];
            v[4] = __uint_as_float(b.x);
            v[5] = __uint_as_float(b.y);
            v[6] = __uint_as_float(b.z);
            v[7] = __uint_as_float(b.w);
        }
    }
};

template <bool kF32>
__device__ __forceinline__ uint2 encode8(const Eight<kF32>& x, float inv) {
    float v[8];
    x.values(v);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)), __NV_SATFINITE, __NV_E4M3);
        w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float block_amax(uint32_t bits) {
    return __uint_as_float(max(bits, 0x0D800000u));  // 2^-100
}

// 1 x 128 blocks: 16 lanes per block; a half warp takes kU neighbouring blocks of one
// row, all loads in flight at once.
template <bool kF32, int kU>
__global__ void __launch_bounds__(256) k_quantize_rows(const void* x, long long ldx, int rows, int cols, uint8_t* codes,
                                                       float* scales) {
    const int kblocks = (cols + 127) / 128;
    const int sub = threadIdx.x & 15;
    const int row = blockIdx.x * 16 + (threadIdx.x >> 4), kb0 = blockIdx.y * kU;
    const int col0 = kb0 * 128 + sub * 8;
    const bool in_rows = row < rows;
    dependent_wait_and_release();
    Eight<kF32> v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        v[u].zero();
        if (in_rows && col0 + u * 128 < cols)
            v[u].load(static_cast<const char*>(x) + (row * ldx + col0 + u * 128) * (kF32 ? 4 : 2));
    }
    float mine = 0.f;  // lane u keeps block u's maximum
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        uint32_t m = v[u].amax();
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float a = block_amax(m);
        if (sub == u) mine = a;
        if (in_rows && col0 + u * 128 < cols)
            *reinterpret_cast<uint2*>(codes + (long long)row * cols + col0 + u * 128) =
                encode8<kF32>(v[u], __fdiv_rn(448.f, a));
    }
    if (in_rows && sub < kU && kb0 + sub < kblocks)
        scales[(long long)row * kblocks + kb0 + sub] = __fdiv_rn(mine, 448.f);
}

// 128 x 128 blocks: one CTA of 512 threads per block, 4 pieces of 8 elements per thread.
template <bool kF32>
__global__ void __launch_bounds__(512) k_quantize_blocks(const void* x, long long ldx, int rows, int cols,
                                                         uint8_t* codes, float* scales) {
    __shared__ uint32_t wmax[16];
    const int kb = blockIdx.x, rb = blockIdx.y;
    const long long mat = blockIdx.z;
    const int col = kb * 128 + (threadIdx.x & 15) * 8;
    Eight<kF32> v[4];
    uint32_t m = 0u;
    dependent_wait_and_release();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = rb * 128 + u * 32 + (threadIdx.x >> 4);
        v[u].zero();
        if (row < rows && col < cols)
            v[u].load(static_cast<const char*>(x) + ((mat * rows + row) * ldx + col) * (kF32 ? 4 : 2));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) m = max(m, v[u].amax());
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) m = max(m, wmax[w]);
    const float a = block_amax(m), inv = __fdiv_rn(448.f, a);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = rb * 128 + u * 32 + (threadIdx.x >> 4);
        if (row < rows && col < cols)
            *reinterpret_cast<uint2*>(codes + (mat * rows + row) * cols + col) = encode8<kF32>(v[u], inv);
    }
    if (threadIdx.x == 0) scales[(mat * gridDim.y + rb) * gridDim.x + kb] = __fdiv_rn(a, 448.f);
}

template <bool kF32>
cudaError_t launch_rows(const void* x, long long ldx, int rows, int cols, uint8_t* codes, float* scales, cudaStream_t s) {
    const int kblocks = (cols + 127) / 128;
    const unsigned gx = (unsigned)((rows + 15) / 16);
    // as many blocks per half warp as a row fills, unless that leaves SMs without work
    // (64 rows of 8192: 6.1 us with four, 4.9 with one)
    if (kblocks >= 4 && (long long)gx * ((kblocks + 3) / 4) >= 2 * tc_num_sms())
        return launch_dependent(k_quantize_rows<kF32, 4>, dim3(gx, (kblocks + 3) / 4), 256, 0, 0, s, x, ldx, rows, cols,
                                codes, scales);
    return launch_dependent(k_quantize_rows<kF32, 1>, dim3(gx, kblocks), 256, 0, 0, s, x, ldx, rows, cols, codes, scales);
}

}  // namespace

cudaError_t launch_quantize_fp8(const void* x, bool f32, long long ldx, int n_mat, int rows, int cols, int block_rows,
                                uint8_t* codes, float* scales, cudaStream_t s) {
    const int kblocks = (cols + 127) / 128;
    if (block_rows == 1) {
        // the matrices' rows follow each other with the same pitch
        return f32 ? launch_rows<true>(x, ldx, n_mat * rows, cols, codes, scales, s)
                   : launch_rows<false>(x, ldx, n_mat * rows, cols, codes, scales, s);
    }
    const dim3 grid(kblocks, (rows + 127) / 128, n_mat);
    return f32 ? launch_dependent(k_quantize_blocks<true>, grid, 512, 0, 0, s, x, ldx, rows, cols, codes, scales)
               : launch_dependent(k_quantize_blocks<false>, grid, 512, 0, 0, s, x, ldx, rows, cols, codes, scales);
}

}  // namespace lmoe
