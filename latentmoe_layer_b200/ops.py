"""Products that need no layer handle, on torch tensors: grouped expert products,
their gradients, the 8-bit quantiser and the block-scaled 8-bit product
(include/latentmoe.h gives formulas, formats and limits).

Argument marshalling only, like the rest of the binding: every function checks
its tensors (ValueError), launches on the current stream of the tensors' device
and raises ``LmoeError`` on a status from the library. Nothing synchronises, no
workspace is kept, and the calls can be captured into a CUDA graph. None of them
records an autograd graph: the gradients are calls of their own.

The smallest calls take about as long to issue as to run, so the checks here
touch each attribute once.
"""
from __future__ import annotations

import torch

from . import LMOE_BF16, LMOE_FP32, LMOE_OK, LmoeError, load

_BF16, _F32, _F8, _I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
_CODE = {_BF16: LMOE_BF16, _F32: LMOE_FP32}
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object


def _fail(where, what):
    raise ValueError("%s: %s" % (where, what))


def _about(t):
    return "%s %s on %s" % (tuple(t.shape), t.dtype, t.device) if isinstance(t, torch.Tensor) else repr(t)


def _pitch(t, rows, cols, name, where):
    """Row pitch of a 2-D tensor whose columns are contiguous and whose rows do not overlap."""
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        _fail(where, "%s's columns must be contiguous and its rows must not overlap (strides %s)" % (name, t.stride()))
    return ld


def _out(where, out, dtype, x, shape):
    """The output, its row pitch and the library's type code."""
    if out is None:
        dtype = dtype or _BF16
        code = _CODE.get(dtype)
        if code is None:
            _fail(where, "the output is bfloat16 or float32, not %s" % dtype)
        return x.new_empty(shape, dtype=dtype), shape[-1], code
    code = _CODE.get(out.dtype)
    if code is None or out.shape != shape or (dtype is not None and out.dtype != dtype) or out.device != x.device:
        _fail(where, "out must be %s%s on %s, got %s" % (shape, " %s" % dtype if dtype else " bfloat16 or float32", x.device,
                                                        _about(out)))
    if len(shape) == 2:
        return out, _pitch(out, shape[0], shape[1], "out", where), code
    if not out.is_contiguous():
        _fail(where, "out must be contiguous (strides %s)" % (out.stride(),))
    return out, shape[-1], code


def _launch(fn, index, sizes, *args):
    """fn(*args, stream) with the tensors' device current, on its current stream. `sizes`: the 32-bit ones among
    the arguments, which ctypes would cut without a word."""
    if max(sizes) > 0x7FFFFFFF:
        _fail(fn, "a size is beyond 2^31 - 1: %s" % (sizes,))
    if torch.cuda.current_device() == index:
        s = getattr(load(), fn)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            s = getattr(load(), fn)(*args, _raw_stream(index))
    if s != LMOE_OK:
        raise LmoeError(s, fn)


def _is(t, dtype, dims, index):
    return t.dtype is dtype and t.dim() == dims and t.get_device() == index


def _explain(where, index, **tensors):
    """Raises for the first tensor that is not as given by name=(tensor, dtype, dims)."""
    for name, (t, dtype, dims) in tensors.items():
        if not isinstance(t, torch.Tensor) or index < 0 or not _is(t, dtype, dims, index):
            _fail(where, "%s must be a %d-D %s tensor on a CUDA device%s, got %s" %
                  (name, dims, dtype, "" if index < 0 else " (%d)" % index, _about(t)))


def grouped_gemm(x, w, counts, out=None, out_dtype=None, zero_tail=False):
    """y[r] = x[r] W[e(r)]^T: x [rows, K] bf16 in expert order, w [E, N, K] bf16,
    counts [E] int32 rows per expert (on the device). Returns y [rows, N] in
    out_dtype (bfloat16 unless given, or out's). Rows behind the last expert's
    keep what they held; zero_tail writes zeros there."""
    index = x.get_device()
    if index < 0 or not (_is(x, _BF16, 2, index) and _is(w, _BF16, 3, index) and _is(counts, _I32, 1, index)):
        _explain("grouped_gemm", index, x=(x, _BF16, 2), w=(w, _BF16, 3), counts=(counts, _I32, 1))
    rows, K = x.shape
    E, N, Kw = w.shape
    if Kw != K or counts.shape[0] != E or not w.is_contiguous() or not counts.is_contiguous():
        _fail("grouped_gemm", "x [rows, K], w [E, N, K] and counts [E] must fit, w and counts contiguous: got %s, %s, %s" %
              (_about(x), _about(w), _about(counts)))
    y, ldy, code = _out("grouped_gemm", out, out_dtype, x, (rows, N))
    _launch("latentmoe_grouped_gemm", index, (E, rows, N, K), x.data_ptr(), _pitch(x, rows, K, "x", "grouped_gemm"), w.data_ptr(),
            counts.data_ptr(), E, rows, N, K, y.data_ptr(), ldy, code, zero_tail)
    return y


def grouped_gemm_dx(dy, w, counts, out=None, out_dtype=None, zero_tail=False):
    """Gradient of grouped_gemm's input: dx[r] = dy[r] W[e(r)], dy [rows, N] bf16.
    Returns dx [rows, K]."""
    index = dy.get_device()
    if index < 0 or not (_is(dy, _BF16, 2, index) and _is(w, _BF16, 3, index) and _is(counts, _I32, 1, index)):
        _explain("grouped_gemm_dx", index, dy=(dy, _BF16, 2), w=(w, _BF16, 3), counts=(counts, _I32, 1))
    rows, N = dy.shape
    E, Nw, K = w.shape
    if Nw != N or counts.shape[0] != E or not w.is_contiguous() or not counts.is_contiguous():
        _fail("grouped_gemm_dx", "dy [rows, N], w [E, N, K] and counts [E] must fit, w and counts contiguous: got %s, %s, %s"
              % (_about(dy), _about(w), _about(counts)))
    dx, lddx, code = _out("grouped_gemm_dx", out, out_dtype, dy, (rows, K))
    _launch("latentmoe_grouped_gemm_dx", index, (E, rows, N, K), dy.data_ptr(), _pitch(dy, rows, N, "dy", "grouped_gemm_dx"), w.data_ptr(),
            counts.data_ptr(), E, rows, N, K, dx.data_ptr(), lddx, code, zero_tail)
    return dx


def grouped_gemm_dw(dy, x, counts, out=None, out_dtype=None):
    """Gradient of grouped_gemm's weights: dW[e] = sum over expert e's rows of
    dy[r]^T x[r]. Returns dw [E, N, K]; an expert without rows gets zeros."""
    index = dy.get_device()
    if index < 0 or not (_is(dy, _BF16, 2, index) and _is(x, _BF16, 2, index) and _is(counts, _I32, 1, index)):
        _explain("grouped_gemm_dw", index, dy=(dy, _BF16, 2), x=(x, _BF16, 2), counts=(counts, _I32, 1))
    rows, N = dy.shape
    rows_x, K = x.shape
    if rows_x != rows or not counts.is_contiguous():
        _fail("grouped_gemm_dw", "dy [rows, N], x [rows, K] and contiguous counts [E] must fit: got %s, %s, %s" %
              (_about(dy), _about(x), _about(counts)))
    E = counts.shape[0]
    dw, _, code = _out("grouped_gemm_dw", out, out_dtype, dy, (E, N, K))
    _launch("latentmoe_grouped_gemm_dw", index, (E, rows, N, K), dy.data_ptr(), _pitch(dy, rows, N, "dy", "grouped_gemm_dw"), x.data_ptr(),
            _pitch(x, rows, K, "x", "grouped_gemm_dw"), counts.data_ptr(), E, rows, N, K, dw.data_ptr(), code)
    return dw


def quantize_fp8(x, block_rows=1):
    """e4m3 codes and fp32 scales of x, bf16 or fp32: [R, K] or [n_mat, R, K] with one
    scale per block_rows x 128 elements. block_rows 1 (activations): scales
    [..., R, ceil(K/128)]; 128 (weights): scales [..., ceil(R/128), ceil(K/128)]."""
    index = x.get_device()
    dims = x.dim()
    code = _CODE.get(x.dtype)
    if block_rows not in (1, 128) or dims not in (2, 3) or code is None or index < 0:
        _fail("quantize_fp8", "x must be a bfloat16 or float32 tensor [R, K] or [n_mat, R, K] on a CUDA device and "
              "block_rows 1 or 128: got %s, %r" % (_about(x), block_rows))
    if dims == 2:
        R, K = x.shape
        n_mat, ldx = 1, _pitch(x, R, K, "x", "quantize_fp8")
        scales = x.new_empty((-(-R // block_rows), -(-K // 128)), dtype=_F32)
    else:
        n_mat, R, K = x.shape
        if not x.is_contiguous():
            _fail("quantize_fp8", "a stack of matrices must be contiguous (strides %s)" % (x.stride(),))
        ldx = K
        scales = x.new_empty((n_mat, -(-R // block_rows), -(-K // 128)), dtype=_F32)
    codes = x.new_empty(x.shape, dtype=_F8)
    _launch("latentmoe_quantize_fp8", index, (n_mat, R, K), x.data_ptr(), ldx, code, n_mat, R, K, block_rows, codes.data_ptr(),
            scales.data_ptr())
    return codes, scales


def gemm_fp8(xq, xs, wq, ws, counts=None, out=None, out_dtype=None, zero_tail=False):
    """y[r, n] = sum over 128-blocks b of xs[r, b] ws[n / 128, b] (xq[r, b] . wq[n, b]),
    with quantize_fp8's codes and scales: xq [rows, K], xs [rows, ceil(K/128)]. Without
    counts wq is [N, K] and ws [ceil(N/128), ceil(K/128)]; with counts [E] int32 the rows
    are in expert order, wq is [E, N, K] and ws [E, ceil(N/128), ceil(K/128)]."""
    index = xq.get_device()
    dims = 2 if counts is None else 3
    if index < 0 or not (_is(xq, _F8, 2, index) and _is(xs, _F32, 2, index) and _is(wq, _F8, dims, index) and
                         _is(ws, _F32, dims, index)):
        _explain("gemm_fp8", index, xq=(xq, _F8, 2), xs=(xs, _F32, 2), wq=(wq, _F8, dims), ws=(ws, _F32, dims))
    rows, K = xq.shape
    kb = -(-K // 128)
    if counts is None:
        E, ptr = 1, None
        N, Kw = wq.shape
        fit = ws.shape == (-(-N // 128), kb)
    else:
        if not _is(counts, _I32, 1, index):
            _explain("gemm_fp8", index, counts=(counts, _I32, 1))
        E, N, Kw = wq.shape
        fit = ws.shape == (E, -(-N // 128), kb) and counts.shape[0] == E and counts.is_contiguous()
        ptr = counts.data_ptr()
    if not fit or Kw != K or xs.shape != (rows, kb) or not (
            xq.is_contiguous() and xs.is_contiguous() and wq.is_contiguous() and ws.is_contiguous()):
        _fail("gemm_fp8", "codes and scales must fit and be contiguous: got xq %s, xs %s, wq %s, ws %s, counts %s" %
              (_about(xq), _about(xs), _about(wq), _about(ws), _about(counts)))
    y, ldy, code = _out("gemm_fp8", out, out_dtype, xq, (rows, N))
    _launch("latentmoe_gemm_fp8", index, (E, rows, N, K), xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), ptr, E, rows, N, K,
            y.data_ptr(), ldy, code, zero_tail)
    return y
