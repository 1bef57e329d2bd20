// ops.cu -- C entry points of the products that need no layer handle: grouped
// products, their gradients, the 8-bit quantiser and the block-scaled 8-bit
// product (include/latentmoe.h). Argument checks, TMA descriptors, one launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "grouped.h"

using namespace lmoe;

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Polls after which a device wait gives up.
std::atomic<unsigned> g_ops_spin{1u << 24};

// What the entry points share, made once per process: the driver's descriptor
// encoder and a pinned word in which kernels count the waits that ran out
// (mapped into every device's address space; the host only reads it, so that
// no report can be taken from the caller it is meant for).
struct OpsState {
    EncodeTiledFn encode = nullptr;
    int* herr = nullptr;
    int* derr = nullptr;
};
std::mutex g_ops_mu;
OpsState g_ops;
std::atomic<bool> g_ops_ready{false};

// An error that is returned is not left behind for a later call's cudaGetLastError.
lmoe_status failed() {
    (void)cudaGetLastError();
    return LMOE_ERR_CUDA;
}

lmoe_status ops_state(const OpsState** out) {
    if (!g_ops_ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_ops_mu);
        if (!g_ops_ready.load(std::memory_order_relaxed)) {
            OpsState st;
            // the first call may come while a stream is being captured: the allocation is not part of the graph
            cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
            if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return failed();
            void* fn = nullptr;
            cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
            bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
                      q == cudaDriverEntryPointSuccess && fn;
            ok = ok && cudaHostAlloc(reinterpret_cast<void**>(&st.herr), 64, cudaHostAllocMapped | cudaHostAllocPortable) ==
                           cudaSuccess;
            ok = ok && cudaHostGetDevicePointer(reinterpret_cast<void**>(&st.derr), st.herr, 0) == cudaSuccess;
            if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) ok = false;
            if (!ok) {
                if (st.herr) cudaFreeHost(st.herr);
                return failed();
            }
            *st.herr = 0;
            st.encode = reinterpret_cast<EncodeTiledFn>(fn);
            g_ops = st;
            g_ops_ready.store(true, std::memory_order_release);
        }
    }
    *out = &g_ops;
    return LMOE_OK;
}

// Waits that ran out since this thread last looked are reported to it once: to every thread,
// as nothing tells which one's launch it was.
lmoe_status take_error(const OpsState& st) {
    thread_local int seen = 0;
    const int now = __atomic_load_n(st.herr, __ATOMIC_ACQUIRE);
    if (now == seen) return LMOE_OK;
    seen = now;
    return LMOE_ERR_TIMEOUT;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline lmoe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? LMOE_OK : failed(); }

// [mats, rows, cols] with a row pitch, boxes of 128 bytes x box_rows, 128-byte
// swizzle; indices past the end are filled with zeros.
bool encode(const OpsState& st, CUtensorMap* m, const void* base, bool bf16, long long mats, long long rows, long long cols,
            long long pitch, int box_rows) {
    const int esz = bf16 ? 2 : 1;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)mats};
    cuuint64_t strides[2] = {(cuuint64_t)(pitch * esz), (cuuint64_t)(pitch * rows * esz)};
    cuuint32_t box[3] = {(cuuint32_t)(128 / esz), (cuuint32_t)box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    auto once = [&] {
        return st.encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                         const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (once()) return true;
    // a host thread that has not used CUDA yet has no context current, which the encoder (a driver
    // call) needs; setting the device it has anyway makes one so
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && once();
}

// The row-side operand [n_rows, cols] in boxes of 128, 64, 32 and 16 rows.
bool encode_rows(const OpsState& st, GgParams& P, const void* base, bool bf16, int n_rows, int cols, long long pitch) {
    for (int i = 0; i < 4; ++i)
        if (!encode(st, &P.b_map[i], base, bf16, 1, n_rows, cols, pitch, 128 >> i)) return false;
    return true;
}

constexpr long long kMaxDim = 1LL << 22;        // N, K
constexpr long long kMaxElems = 1LL << 38;      // elements of one operand
constexpr long long kMaxTiles = 1LL << 30;      // tiles of one launch
constexpr int kMaxRows = 1 << 30;               // row indices and their tiles' ends stay inside 32 bits
constexpr long long kMaxRowBlocks = 0x7FFFFFF0; // of the quantiser: rows rounded up to its 16 per CTA stay inside 32 bits

// Sizes of a product: n_rows rows in n_groups groups, weights [n_groups, N, K].
lmoe_status check_sizes(int n_groups, int n_rows, int N, int K, int k_align) {
    if (n_groups <= 0 || n_rows < 0 || N <= 0 || K <= 0) return LMOE_ERR_INVALID_ARG;
    if (n_groups > kMaxE || n_rows > kMaxRows || N % 8 || K % k_align || N > kMaxDim || K > kMaxDim)
        return LMOE_ERR_UNSUPPORTED;
    if ((long long)n_groups * N > kMaxElems / K) return LMOE_ERR_UNSUPPORTED;
    const long long side = N > K ? N : K;
    if (((long long)n_rows / 256 + n_groups + 1) * ((side + 255) / 256) > kMaxTiles ||
        (long long)n_groups * ((N + 255) / 256) * ((K + 255) / 256) > kMaxTiles)
        return LMOE_ERR_UNSUPPORTED;
    return LMOE_OK;
}
// A row-major operand: 16-byte aligned base and rows, no overlapping rows. A
// matrix without rows has no address to check.
lmoe_status check_rows(const void* p, long long ld, int n_rows, int cols, int align_elems) {
    if (n_rows == 0) return LMOE_OK;
    if (!p || !aligned(p, 16) || ld < cols || ld % align_elems) return LMOE_ERR_INVALID_ARG;
    if (ld > kMaxElems / n_rows) return LMOE_ERR_UNSUPPORTED;
    return LMOE_OK;
}
lmoe_status check_counts(const int32_t* counts) {
    return counts && aligned(counts, 4) ? LMOE_OK : LMOE_ERR_INVALID_ARG;
}
bool is_out_type(lmoe_dtype t) { return t == LMOE_BF16 || t == LMOE_FP32; }

// Contraction accumulated in TMEM before it is added into fp32 registers, in
// 64-deep k-blocks: 512 deep for fp32 outputs, 4096 for bf16 outputs. The tensor
// core's additions err towards zero: like-signed sums of 2^22 products, never
// drained, came out 2.4% low.
int chunk_blocks(lmoe_dtype out) { return out == LMOE_FP32 ? 8 : 64; }

GgParams base_params(const OpsState& st, const int32_t* counts, int n_groups, int n_rows, lmoe_dtype out_type) {
    GgParams P;
    memset(&P, 0, sizeof(P));
    P.counts = counts;
    P.n_groups = n_groups;
    P.n_rows = n_rows;
    P.out_f32 = out_type == LMOE_FP32;
    P.chunk_kb = chunk_blocks(out_type);
    P.err = st.derr;
    P.spin = g_ops_spin.load(std::memory_order_relaxed);
    return P;
}

// y [n_rows, N] = x W^T (dx = false) or dx [n_rows, K] = dy W (dx = true).
lmoe_status run_rows(bool dx, const void* a, long long lda, const void* w, const int32_t* counts, int n_groups, int n_rows,
                     int N, int K, void* out, long long ldo, lmoe_dtype out_type, int zero_tail, void* stream) {
    lmoe_status s = check_sizes(n_groups, n_rows, N, K, 8);
    if (s != LMOE_OK) return s;
    const int in_cols = dx ? N : K, out_cols = dx ? K : N;
    if (!is_out_type(out_type) || !w || !aligned(w, 16)) return LMOE_ERR_INVALID_ARG;
    if ((s = check_counts(counts)) != LMOE_OK || (s = check_rows(a, lda, n_rows, in_cols, 8)) != LMOE_OK ||
        (s = check_rows(out, ldo, n_rows, out_cols, 8)) != LMOE_OK)
        return s;
    if (n_rows == 0) return LMOE_OK;
    const OpsState* st = nullptr;
    if ((s = ops_state(&st)) != LMOE_OK || (s = take_error(*st)) != LMOE_OK) return s;
    GgParams P = base_params(*st, counts, n_groups, n_rows, out_type);
    P.out = out;
    P.ldo = ldo;
    P.feat = out_cols;
    P.cdim = in_cols;
    P.zero_tail = zero_tail != 0;
    if (!dx && n_rows <= kFewRows)
        return cuda_status(launch_few(false, w, a, lda * 2, P, static_cast<cudaStream_t>(stream)));
    if (!encode(*st, &P.a_map, w, true, n_groups, N, K, K, dx ? 64 : 128) ||
        !encode_rows(*st, P, a, true, n_rows, in_cols, lda))
        return failed();
    return cuda_status(launch_grouped(dx ? GG_DX : GG_FWD, P, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

lmoe_status latentmoe_grouped_gemm(const void* x, long long ldx, const void* w, const int32_t* counts, int n_groups,
                                   int n_rows, int N, int K, void* y, long long ldy, lmoe_dtype y_dtype, int zero_tail,
                                   void* stream) {
    return run_rows(false, x, ldx, w, counts, n_groups, n_rows, N, K, y, ldy, y_dtype, zero_tail, stream);
}

lmoe_status latentmoe_grouped_gemm_dx(const void* dy, long long lddy, const void* w, const int32_t* counts, int n_groups,
                                      int n_rows, int N, int K, void* dx, long long lddx, lmoe_dtype dx_dtype,
                                      int zero_tail, void* stream) {
    return run_rows(true, dy, lddy, w, counts, n_groups, n_rows, N, K, dx, lddx, dx_dtype, zero_tail, stream);
}

lmoe_status latentmoe_grouped_gemm_dw(const void* dy, long long lddy, const void* x, long long ldx, const int32_t* counts,
                                      int n_groups, int n_rows, int N, int K, void* dw, lmoe_dtype dw_dtype,
                                      void* stream) {
    lmoe_status s = check_sizes(n_groups, n_rows, N, K, 8);
    if (s != LMOE_OK) return s;
    if (!is_out_type(dw_dtype) || !dw || !aligned(dw, 16)) return LMOE_ERR_INVALID_ARG;
    if ((s = check_counts(counts)) != LMOE_OK || (s = check_rows(dy, lddy, n_rows, N, 8)) != LMOE_OK ||
        (s = check_rows(x, ldx, n_rows, K, 8)) != LMOE_OK)
        return s;
    const OpsState* st = nullptr;
    if ((s = ops_state(&st)) != LMOE_OK || (s = take_error(*st)) != LMOE_OK) return s;
    if (n_rows == 0)  // no rows anywhere: every gradient is zero
        return cuda_status(cudaMemsetAsync(dw, 0, (size_t)n_groups * N * K * (dw_dtype == LMOE_FP32 ? 4 : 2),
                                           static_cast<cudaStream_t>(stream)));
    GgParams P = base_params(*st, counts, n_groups, n_rows, dw_dtype);
    P.out = dw;
    P.ldo = K;
    P.feat = K;
    P.cols = N;
    if (!encode(*st, &P.a_map, x, true, 1, n_rows, K, ldx, 64) || !encode(*st, &P.b_map[0], dy, true, 1, n_rows, N, lddy, 64))
        return failed();
    return cuda_status(launch_grouped(GG_DW, P, static_cast<cudaStream_t>(stream)));
}

lmoe_status latentmoe_quantize_fp8(const void* x, long long ldx, lmoe_dtype x_dtype, int n_mat, int R, int K,
                                   int block_rows, void* codes, float* scales, void* stream) {
    if (n_mat < 0 || R < 0 || K <= 0 || !is_out_type(x_dtype) || (block_rows != 1 && block_rows != 128))
        return LMOE_ERR_INVALID_ARG;
    if (n_mat == 0 || R == 0) return LMOE_OK;
    if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || ldx < K)
        return LMOE_ERR_INVALID_ARG;
    if (ldx % (x_dtype == LMOE_FP32 ? 4 : 8)) return LMOE_ERR_INVALID_ARG;
    if (K % 16 || K > kMaxDim || n_mat > 65535 || (block_rows == 128 && R > 65535 * 128)) return LMOE_ERR_UNSUPPORTED;
    const long long rows = (long long)n_mat * R;
    if (ldx > kMaxElems / rows || rows * ((K + 127) / 128) > kMaxRowBlocks) return LMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_quantize_fp8(x, x_dtype == LMOE_FP32, ldx, n_mat, R, K, block_rows,
                                           static_cast<uint8_t*>(codes), scales, static_cast<cudaStream_t>(stream)));
}

lmoe_status latentmoe_gemm_fp8(const void* xq, const float* xs, const void* wq, const float* ws, const int32_t* counts,
                               int n_groups, int n_rows, int N, int K, void* y, long long ldy, lmoe_dtype y_dtype,
                               int zero_tail, void* stream) {
    lmoe_status s = check_sizes(n_groups, n_rows, N, K, 16);
    if (s != LMOE_OK) return s;
    if (!is_out_type(y_dtype) || !wq || !aligned(wq, 16) || !ws || !aligned(ws, 16)) return LMOE_ERR_INVALID_ARG;
    if (counts ? !aligned(counts, 4) : n_groups != 1) return LMOE_ERR_INVALID_ARG;
    if (n_rows && (!xs || !aligned(xs, 16))) return LMOE_ERR_INVALID_ARG;
    if ((s = check_rows(xq, K, n_rows, K, 16)) != LMOE_OK || (s = check_rows(y, ldy, n_rows, N, 8)) != LMOE_OK) return s;
    if (n_rows == 0) return LMOE_OK;
    const OpsState* st = nullptr;
    if ((s = ops_state(&st)) != LMOE_OK || (s = take_error(*st)) != LMOE_OK) return s;
    GgParams P = base_params(*st, counts, n_groups, n_rows, y_dtype);
    P.a_scale = ws;
    P.b_scale = xs;
    P.out = y;
    P.ldo = ldy;
    P.feat = N;
    P.cdim = K;
    P.zero_tail = zero_tail != 0;
    if (n_rows <= kFewRows)
        return cuda_status(launch_few(true, wq, xq, K, P, static_cast<cudaStream_t>(stream)));
    if (!encode(*st, &P.a_map, wq, false, n_groups, N, K, K, 128) ||
        !encode_rows(*st, P, xq, false, n_rows, K, K))
        return failed();
    const int op = n_rows / n_groups > 64 ? GG_FP8_ROWS : GG_FP8;
    return cuda_status(launch_grouped(op, P, static_cast<cudaStream_t>(stream)));
}

lmoe_status latentmoe_products_status(void) {
    return g_ops_ready.load(std::memory_order_acquire) ? take_error(g_ops) : LMOE_OK;
}

lmoe_status latentmoe_set_products_wait_limit(long long polls) {
    if (polls < 0 || polls > 0xFFFFFFFFLL) return LMOE_ERR_INVALID_ARG;
    g_ops_spin.store((unsigned)polls, std::memory_order_relaxed);
    return LMOE_OK;
}

}  // extern "C"
