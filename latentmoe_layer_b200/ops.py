"""Products that need no layer handle, on torch tensors: grouped expert products,
their gradients, the 8-bit quantiser and the block-scaled 8-bit product
(include/latentmoe.h gives formulas, formats and limits).

Argument marshalling only, like the rest of the binding: every function checks
its tensors (ValueError), launches on the current stream of the tensors' device
and raises ``LmoeError`` on a status from the library. Nothing synchronises, no
workspace is kept, and the calls can be captured into a CUDA graph. None of them
records an autograd graph: the gradients are calls of their own.
"""
from __future__ import annotations

import ctypes

_void = ctypes.c_void_p


def _fail(where, what):
    raise ValueError("%s: %s" % (where, what))


def _rows(t, name, where, dtypes):
    """Row pitch of a 2-D tensor whose columns are contiguous."""
    if t.dim() != 2 or t.dtype not in dtypes:
        _fail(where, "%s must be a 2-D tensor of %s, got %s %s" % (name, "/".join(map(str, dtypes)), tuple(t.shape), t.dtype))
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        _fail(where, "%s's columns must be contiguous (strides %s)" % (name, t.stride()))
    if rows <= 1:
        return cols
    ld = t.stride(0)
    if ld < cols:
        _fail(where, "%s's rows overlap (strides %s)" % (name, t.stride()))
    return ld


def _same_device(where, first, **others):
    if not first.is_cuda:
        _fail(where, "the tensors must be on a CUDA device")
    for name, t in others.items():
        if t is not None and t.device != first.device:
            _fail(where, "%s is on %s, not on %s" % (name, t.device, first.device))


def _counts(counts, groups, where):
    import torch
    if counts.dim() != 1 or counts.dtype != torch.int32 or counts.shape[0] != groups or not counts.is_contiguous():
        _fail(where, "counts must be a contiguous int32 tensor [%d], got %s %s" % (groups, tuple(counts.shape), counts.dtype))


def _out(out, shape, dtype, device, where):
    """The output tensor, its row pitch and the library's type code."""
    import torch
    if out is None:
        if dtype not in (torch.bfloat16, torch.float32):
            _fail(where, "the output is bfloat16 or float32, not %s" % dtype)
        out = torch.empty(shape, dtype=dtype, device=device)
    else:
        if tuple(out.shape) != tuple(shape) or (dtype is not None and out.dtype != dtype):
            _fail(where, "out must be %s%s, got %s %s" % (tuple(shape), "" if dtype is None else " %s" % dtype,
                                                         tuple(out.shape), out.dtype))
        if out.device != device:
            _fail(where, "out is on %s, not on %s" % (out.device, device))
    if len(shape) == 2:
        ld = _rows(out, "out", where, (torch.bfloat16, torch.float32))
    else:
        if out.dtype not in (torch.bfloat16, torch.float32) or not out.is_contiguous():
            _fail(where, "out must be a contiguous bfloat16 or float32 tensor")
        ld = shape[-1]
    return out, ld, 1 if out.dtype == torch.float32 else 0


def _call(name, device, *args):
    """Launches lib.name(*args, stream) with `device` current."""
    import torch
    from . import LMOE_OK, LmoeError, load
    fn = getattr(load(), name)
    stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        s = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            s = fn(*args, stream)
    if s != LMOE_OK:
        raise LmoeError(s, name)


def _weights(w, where):
    import torch
    if w.dim() != 3 or w.dtype != torch.bfloat16 or not w.is_contiguous():
        _fail(where, "w must be a contiguous bfloat16 tensor [E, N, K], got %s %s" % (tuple(w.shape), w.dtype))
    return w.shape


def grouped_gemm(x, w, counts, out=None, out_dtype=None, zero_tail=False):
    """y[r] = x[r] W[e(r)]^T: x [rows, K] bf16 in expert order, w [E, N, K] bf16,
    counts [E] int32 rows per expert (on the device). Returns y [rows, N] in
    out_dtype (bfloat16 unless given, or out's). Rows behind the last expert's
    keep what they held; zero_tail writes zeros there."""
    import torch
    where = "grouped_gemm"
    E, N, K = _weights(w, where)
    _same_device(where, x, w=w, counts=counts)
    ldx = _rows(x, "x", where, (torch.bfloat16,))
    if x.shape[1] != K:
        _fail(where, "x has %d columns, w %d" % (x.shape[1], K))
    _counts(counts, E, where)
    rows = x.shape[0]
    y, ldy, code = _out(out, (rows, N), out_dtype or (torch.bfloat16 if out is None else None), x.device, where)
    _call("latentmoe_grouped_gemm", x.device, x.data_ptr(), ldx, w.data_ptr(), counts.data_ptr(), E, rows, N, K,
          y.data_ptr(), ldy, code, int(zero_tail))
    return y


def grouped_gemm_dx(dy, w, counts, out=None, out_dtype=None, zero_tail=False):
    """Gradient of grouped_gemm's input: dx[r] = dy[r] W[e(r)], dy [rows, N] bf16.
    Returns dx [rows, K]."""
    import torch
    where = "grouped_gemm_dx"
    E, N, K = _weights(w, where)
    _same_device(where, dy, w=w, counts=counts)
    lddy = _rows(dy, "dy", where, (torch.bfloat16,))
    if dy.shape[1] != N:
        _fail(where, "dy has %d columns, w %d rows" % (dy.shape[1], N))
    _counts(counts, E, where)
    rows = dy.shape[0]
    dx, lddx, code = _out(out, (rows, K), out_dtype or (torch.bfloat16 if out is None else None), dy.device, where)
    _call("latentmoe_grouped_gemm_dx", dy.device, dy.data_ptr(), lddy, w.data_ptr(), counts.data_ptr(), E, rows, N, K,
          dx.data_ptr(), lddx, code, int(zero_tail))
    return dx


def grouped_gemm_dw(dy, x, counts, out=None, out_dtype=None):
    """Gradient of grouped_gemm's weights: dW[e] = sum over expert e's rows of
    dy[r]^T x[r]. Returns dw [E, N, K]; an expert without rows gets zeros."""
    import torch
    where = "grouped_gemm_dw"
    _same_device(where, dy, x=x, counts=counts)
    lddy = _rows(dy, "dy", where, (torch.bfloat16,))
    ldx = _rows(x, "x", where, (torch.bfloat16,))
    rows, N = dy.shape
    if x.shape[0] != rows:
        _fail(where, "dy has %d rows, x %d" % (rows, x.shape[0]))
    K = x.shape[1]
    E = counts.shape[0] if counts.dim() == 1 else -1
    _counts(counts, E, where)
    dw, _, code = _out(out, (E, N, K), out_dtype or (torch.bfloat16 if out is None else None), dy.device, where)
    _call("latentmoe_grouped_gemm_dw", dy.device, dy.data_ptr(), lddy, x.data_ptr(), ldx, counts.data_ptr(), E, rows, N, K,
          dw.data_ptr(), code)
    return dw


def quantize_fp8(x, block_rows=1):
    """e4m3 codes and fp32 scales of x, bf16 or fp32: [R, K] or [n_mat, R, K] with one
    scale per block_rows x 128 elements. block_rows 1 (activations): scales
    [..., R, ceil(K/128)]; 128 (weights): scales [..., ceil(R/128), ceil(K/128)]."""
    import torch
    where = "quantize_fp8"
    if block_rows not in (1, 128):
        _fail(where, "block_rows is 1 or 128, not %r" % (block_rows,))
    if x.dim() not in (2, 3) or x.dtype not in (torch.bfloat16, torch.float32):
        _fail(where, "x must be a bfloat16 or float32 tensor [R, K] or [n_mat, R, K], got %s %s" % (tuple(x.shape), x.dtype))
    _same_device(where, x)
    n_mat = x.shape[0] if x.dim() == 3 else 1
    R, K = x.shape[-2:]
    if x.dim() == 3:
        if not x.is_contiguous():
            _fail(where, "x must be contiguous (strides %s)" % (x.stride(),))
        ldx = K
    else:
        ldx = _rows(x, "x", where, (torch.bfloat16, torch.float32))
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((*x.shape[:-2], -(-R // block_rows), -(-K // 128)), dtype=torch.float32, device=x.device)
    _call("latentmoe_quantize_fp8", x.device, x.data_ptr(), ldx, 1 if x.dtype == torch.float32 else 0, n_mat, R, K,
          block_rows, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def gemm_fp8(xq, xs, wq, ws, counts=None, out=None, out_dtype=None, zero_tail=False):
    """y[r, n] = sum over 128-blocks b of xs[r, b] ws[n / 128, b] (xq[r, b] . wq[n, b]),
    with quantize_fp8's codes and scales: xq [rows, K], xs [rows, ceil(K/128)]. Without
    counts wq is [N, K] and ws [ceil(N/128), ceil(K/128)]; with counts [E] int32 the rows
    are in expert order, wq is [E, N, K] and ws [E, ceil(N/128), ceil(K/128)]."""
    import torch
    where = "gemm_fp8"
    f8 = torch.float8_e4m3fn
    lead = 0 if counts is None else 1
    if wq.dim() != 2 + lead or wq.dtype != f8 or not wq.is_contiguous():
        _fail(where, "wq must be a contiguous float8_e4m3fn tensor %s, got %s %s" %
              ("[N, K]" if counts is None else "[E, N, K]", tuple(wq.shape), wq.dtype))
    E = wq.shape[0] if lead else 1
    N, K = wq.shape[-2:]
    kb = -(-K // 128)
    _same_device(where, xq, xs=xs, wq=wq, ws=ws, counts=counts)
    if xq.dim() != 2 or xq.dtype != f8 or not xq.is_contiguous() or xq.shape[1] != K:
        _fail(where, "xq must be a contiguous float8_e4m3fn tensor [rows, %d], got %s %s" % (K, tuple(xq.shape), xq.dtype))
    rows = xq.shape[0]
    for name, t, shape in (("xs", xs, (rows, kb)), ("ws", ws, (*wq.shape[:-2], -(-N // 128), kb))):
        if tuple(t.shape) != tuple(shape) or t.dtype != torch.float32 or not t.is_contiguous():
            _fail(where, "%s must be a contiguous float32 tensor %s, got %s %s" % (name, tuple(shape), tuple(t.shape), t.dtype))
    if counts is not None:
        _counts(counts, E, where)
    y, ldy, code = _out(out, (rows, N), out_dtype or (torch.bfloat16 if out is None else None), xq.device, where)
    _call("latentmoe_gemm_fp8", xq.device, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
          None if counts is None else counts.data_ptr(), E, rows, N, K, y.data_ptr(), ldy, code, int(zero_tail))
    return y
