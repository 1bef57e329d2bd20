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

__device__ __forceinline__ uint32_t max_bits(uint32_t m, float v) {
    return max(m, __float_as_uint(v) & 0x7FFFFFFFu);
}

// Eight elements from p (16-byte aligned).
template <bool kF32>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
    if (kF32) {
        const uint4 a = ld_global_nc_v4(static_cast<const uint4*>(p)), b = ld_global_nc_v4(static_cast<const uint4*>(p) + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        const uint4 a = ld_global_nc_v4(static_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
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

// 1 x 128 blocks: 16 lanes per block, kUnroll blocks per half warp in flight.
template <bool kF32>
__global__ void __launch_bounds__(256) k_quantize_rows(const void* x, long long ldx, long long rows, int cols,
                                                       uint8_t* codes, float* scales) {
    constexpr int kUnroll = kF32 ? 2 : 4;
    const int kblocks = (cols + 127) / 128;
    const long long total = rows * kblocks;
    const int sub = threadIdx.x & 15;
    const long long first = (long long)(blockIdx.x * (blockDim.x / 16) + threadIdx.x / 16) * kUnroll;
    float v[kUnroll][8];
    uint32_t m[kUnroll];
    long long row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const long long b = first + u;
        row[u] = b / kblocks;
        col[u] = (int)(b - row[u] * kblocks) * 128 + sub * 8;
        const bool in = b < total && col[u] < cols;
        if (!in) col[u] = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (in) load8<kF32>(static_cast<const char*>(x) + (row[u] * ldx + col[u]) * (kF32 ? 4 : 2), v[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        m[u] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[u] = max_bits(m[u], v[u][i]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[u] = max(m[u], __shfl_xor_sync(0xFFFFFFFFu, m[u], o));
        const float a = block_amax(m[u]);
        if (col[u] >= 0) {
            *reinterpret_cast<uint2*>(codes + row[u] * cols + col[u]) = encode8(v[u], __fdiv_rn(448.f, a));
            if (sub == 0) scales[first + u] = __fdiv_rn(a, 448.f);
        }
    }
}

// 128 x 128 blocks: one CTA of 512 threads per block, 4 pieces of 8 elements per thread.
template <bool kF32>
__global__ void __launch_bounds__(512) k_quantize_blocks(const void* x, long long ldx, int rows, int cols,
                                                         uint8_t* codes, float* scales) {
    __shared__ uint32_t wmax[16];
    const int kb = blockIdx.x, rb = blockIdx.y;
    const long long mat = blockIdx.z;
    const int col = kb * 128 + (threadIdx.x & 15) * 8;
    float v[4][8];
    uint32_t m = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = rb * 128 + u * 32 + (threadIdx.x >> 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (row < rows && col < cols)
            load8<kF32>(static_cast<const char*>(x) + ((mat * rows + row) * ldx + col) * (kF32 ? 4 : 2), v[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_bits(m, v[u][i]);
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
            *reinterpret_cast<uint2*>(codes + (mat * rows + row) * cols + col) = encode8(v[u], inv);
    }
    if (threadIdx.x == 0) scales[(mat * gridDim.y + rb) * gridDim.x + kb] = __fdiv_rn(a, 448.f);
}

}  // namespace

cudaError_t launch_quantize_fp8(const void* x, bool f32, long long ldx, int n_mat, int rows, int cols, int block_rows,
                                uint8_t* codes, float* scales, cudaStream_t s) {
    const int kblocks = (cols + 127) / 128;
    if (block_rows == 1) {
        const long long nrows = (long long)n_mat * rows;
        const long long per = 16 * (f32 ? 2 : 4);  // blocks per CTA
        const long long grid = (nrows * kblocks + per - 1) / per;
        if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
        if (f32) k_quantize_rows<true><<<(unsigned)grid, 256, 0, s>>>(x, ldx, nrows, cols, codes, scales);
        else k_quantize_rows<false><<<(unsigned)grid, 256, 0, s>>>(x, ldx, nrows, cols, codes, scales);
    } else {
        const dim3 grid(kblocks, (rows + 127) / 128, n_mat);
        if (f32) k_quantize_blocks<true><<<grid, 512, 0, s>>>(x, ldx, rows, cols, codes, scales);
        else k_quantize_blocks<false><<<grid, 512, 0, s>>>(x, ldx, rows, cols, codes, scales);
    }
    return cudaGetLastError();
}

}  // namespace lmoe
