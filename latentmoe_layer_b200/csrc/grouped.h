// grouped.h -- parameters and launchers of the grouped products and of the
// block-scaled 8-bit quantiser.
#pragma once
#include "lmoe_internal.h"

namespace lmoe {

enum GgOp : int { GG_FWD = 0, GG_DX = 1, GG_DW = 2, GG_FP8 = 3, GG_FP8_ROWS = 4 };

struct alignas(64) GgParams {
    CUtensorMap a_map;    // feature-side operand
    CUtensorMap b_map[4]; // row-side operand, boxes of 128, 64, 32 and 16 rows (GG_DW: the first, 64 x 64)
    const int* counts;    // [n_groups] rows per group; null: one group of n_rows rows
    const float* a_scale; // GG_FP8: [n_groups, ceil(feat / 128), ceil(cdim / 128)]
    const float* b_scale; // GG_FP8: [n_rows, ceil(cdim / 128)]
    void* out;
    long long ldo;        // output row pitch, elements
    int n_groups, n_rows;
    int feat;             // output columns (the MMA's M side)
    int cdim;             // contraction length (GG_DW: the group's rows instead)
    int cols;             // GG_DW: rows of each dW[e]
    int out_f32;
    int zero_tail;        // 1: rows behind the last group are written as zeros
    int chunk_kb;         // k-blocks per TMEM chunk (8-bit: set by the tile)
    int splits;           // set by launch_grouped: pairs (a cluster of them) that share a tile's contraction
    int* err;             // counts waits that ran out, for the host; never read by a kernel
    unsigned spin;        // polls after which a wait runs out
};

// Launches a kernel as a dependent of the one before it in the stream: its launch and
// set-up run under that kernel's end (dependent_wait_and_release in ptx.cuh). cluster 0: none.
template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);  // this launch's error, no earlier call's
}

// GG_FWD (f8 = false) and GG_FP8 for up to kFewRows rows, where the kernel that splits a matrix over
// all SMs is the faster one (few.cu has both sides' times); P's tensor maps are not used.
constexpr int kFewRows = 8;
cudaError_t launch_few(bool f8, const void* w, const void* x, long long ldx_bytes, const GgParams& P, cudaStream_t s);
cudaError_t launch_grouped(int op, const GgParams& P, cudaStream_t s);
cudaError_t launch_quantize_fp8(const void* x, bool f32, long long ldx, int n_mat, int rows, int cols, int block_rows,
                                uint8_t* codes, float* scales, cudaStream_t s);

}  // namespace lmoe
