"""Products that need no layer handle, on torch tensors: grouped expert products,
their gradients, the 8-bit quantiser and the block-scaled 8-bit product
(include/latentmoe.h gives formulas, formats and limits).

Argument marshalling only, like the rest of the binding: every function checks
its tensors (ValueError), launches on the current stream of the tensors' device
and raises ``LmoeError`` on a status from the library. Nothing synchronises, no
workspace is kept, and the calls can be captured into a CUDA graph.

``grouped_gemm`` is differentiable once, in x and w. The others record no autograd
graph: the gradients are there to be called, and 8-bit codes have none. A write to
``out`` is known to autograd (its version counts up).

The smallest calls take longer to issue than to run (8 us against 4), so the
checks touch each attribute once, in one expression, and the text of a refusal
is put together afterwards.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import LMOE_BF16, LMOE_FP32, LMOE_OK, LmoeError, load

_BF16, _F32, _F8, _I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
_CODE = {_BF16: LMOE_BF16, _F32: LMOE_FP32}
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object
_current_device = torch._C._cuda_getDevice  # a tensor on the device has initialised CUDA
_MAX = 0x7FFFFFFF


def _about(t):
    return "%s %s on %s" % (tuple(t.shape), t.dtype, t.device) if isinstance(t, torch.Tensor) else repr(t)


def _refuse(where, wanted, *tensors):
    raise ValueError("%s: %s, got %s" % (where, wanted, "; ".join(map(_about, tensors))))


def _pitch(t, rows, cols, name, where):
    """Row pitch of a 2-D tensor whose columns are contiguous and whose rows do not overlap."""
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError("%s: %s's columns must be contiguous and its rows must not overlap (strides %s)" %
                         (where, name, t.stride()))
    return ld


def _out(where, out, dtype, x, shape):
    """The output, its row pitch and the library's type code."""
    if out is None:
        code = LMOE_BF16 if dtype is None else _CODE.get(dtype)
        if code is None:
            raise ValueError("%s: the output is bfloat16 or float32, not %s" % (where, dtype))
        return x.new_empty(*shape, dtype=dtype or _BF16), shape[-1], code  # a tuple takes 0.9 us longer to parse
    code = _CODE.get(out.dtype)
    if code is None or out.shape != shape or (dtype is not None and out.dtype != dtype) or out.device != x.device:
        _refuse(where, "out must be %s%s on %s" % (shape, " %s" % dtype if dtype else " bfloat16 or float32", x.device), out)
    if len(shape) == 2:
        return out, _pitch(out, shape[0], shape[1], "out", where), code
    if not out.is_contiguous():
        raise ValueError("%s: out must be contiguous (strides %s)" % (where, out.stride()))
    return out, shape[-1], code


def _written(out):
    """Autograd hears of a write that it did not make."""
    if not out.is_inference():
        increment_version(out)


def _launch(fn, index, *args):
    """fn(*args, stream) with the tensors' device current, on its current stream."""
    if _current_device() == index:
        s = getattr(load(), fn)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            s = getattr(load(), fn)(*args, _raw_stream(index))
    if s != LMOE_OK:
        raise LmoeError(s, fn)


def _too_large(where, *sizes):
    """The library's sizes are 32 bits wide, and ctypes would cut longer ones without a word."""
    raise ValueError("%s: a size is beyond 2^31 - 1: %s" % (where, sizes))


_GROUPED = "x [rows, K] bfloat16, contiguous w [E, N, K] bfloat16 and contiguous counts [E] int32 on one CUDA device"
_DX = "dy [rows, N] bfloat16, contiguous w [E, N, K] bfloat16 and contiguous counts [E] int32 on one CUDA device"
_DW = "dy [rows, N] and x [rows, K] bfloat16 and contiguous counts [E] int32 on one CUDA device"
_QUANT = "x [R, K] or contiguous [n_mat, R, K], bfloat16 or float32, on a CUDA device, and block_rows 1 or 128"
_DENSE8 = "contiguous xq [rows, K] and wq [N, K] float8_e4m3fn, xs [rows, K/128] and ws [N/128, K/128] float32 (rounded " \
          "up) on one CUDA device"
_GROUPED8 = "contiguous xq [rows, K] and wq [E, N, K] float8_e4m3fn, xs [rows, K/128] and ws [E, N/128, K/128] float32 " \
            "(rounded up), counts [E] int32 on one CUDA device"


def grouped_gemm(x, w, counts, out=None, out_dtype=None, zero_tail=False):
    """y[r] = x[r] W[e(r)]^T: x [rows, K] bf16 in expert order, w [E, N, K] bf16,
    counts [E] int32 rows per expert (on the device). Returns y [rows, N] in
    out_dtype (bfloat16 unless given, or out's). Rows behind the last expert's
    keep what they held; zero_tail writes zeros there.

    Where x or w requires a gradient it is recorded (not with out=, which is refused
    then): backward gives dx, zeros behind the last expert, and dw, both bfloat16."""
    if (x.requires_grad or w.requires_grad) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("grouped_gemm: out= records no gradient, and x or w requires one (use torch.no_grad())")
        return _GroupedGemm.apply(x, w, counts, out_dtype, zero_tail)
    index = x.get_device()
    if (index < 0 or x.dtype is not _BF16 or x.dim() != 2 or w.dtype is not _BF16 or w.dim() != 3 or counts.dtype is not _I32
            or counts.dim() != 1 or w.get_device() != index or counts.get_device() != index or not w.is_contiguous()
            or not counts.is_contiguous()):
        _refuse("grouped_gemm", _GROUPED, x, w, counts)
    rows, K = x.shape
    E, N, Kw = w.shape
    if Kw != K or counts.numel() != E:
        _refuse("grouped_gemm", _GROUPED, x, w, counts)
    if (E | rows | N | K) > _MAX:
        _too_large("grouped_gemm", E, rows, N, K)
    y, ldy, code = _out("grouped_gemm", out, out_dtype, x, (rows, N))
    ldx = K if x.is_contiguous() else _pitch(x, rows, K, "x", "grouped_gemm")
    _launch("latentmoe_grouped_gemm", index, x.data_ptr(), ldx, w.data_ptr(), counts.data_ptr(), E, rows, N, K,
            y.data_ptr(), ldy, code, zero_tail)
    if out is not None:
        _written(out)
    return y


class _GroupedGemm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, counts, out_dtype, zero_tail):
        ctx.save_for_backward(x, w, counts)
        return grouped_gemm(x, w, counts, out_dtype=out_dtype, zero_tail=zero_tail)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, counts = ctx.saved_tensors
        # of any strides (sum() hands down strides of 0), and fp32 for an fp32 output: the products
        # read bf16, so that gradient is rounded once, as bf16 activations' are
        dy = dy.to(_BF16).contiguous()
        if dy.data_ptr() % 16:
            dy = dy.clone()
        dx = grouped_gemm_dx(dy, w, counts, zero_tail=True) if ctx.needs_input_grad[0] else None
        dw = grouped_gemm_dw(dy, x, counts) if ctx.needs_input_grad[1] else None
        return dx, dw, None, None, None


def grouped_gemm_dx(dy, w, counts, out=None, out_dtype=None, zero_tail=False):
    """Gradient of grouped_gemm's input: dx[r] = dy[r] W[e(r)], dy [rows, N] bf16.
    Returns dx [rows, K]."""
    index = dy.get_device()
    if (index < 0 or dy.dtype is not _BF16 or dy.dim() != 2 or w.dtype is not _BF16 or w.dim() != 3
            or counts.dtype is not _I32 or counts.dim() != 1 or w.get_device() != index or counts.get_device() != index
            or not w.is_contiguous() or not counts.is_contiguous()):
        _refuse("grouped_gemm_dx", _DX, dy, w, counts)
    rows, N = dy.shape
    E, Nw, K = w.shape
    if Nw != N or counts.numel() != E:
        _refuse("grouped_gemm_dx", _DX, dy, w, counts)
    if (E | rows | N | K) > _MAX:
        _too_large("grouped_gemm_dx", E, rows, N, K)
    dx, lddx, code = _out("grouped_gemm_dx", out, out_dtype, dy, (rows, K))
    lddy = N if dy.is_contiguous() else _pitch(dy, rows, N, "dy", "grouped_gemm_dx")
    _launch("latentmoe_grouped_gemm_dx", index, dy.data_ptr(), lddy, w.data_ptr(), counts.data_ptr(), E, rows, N, K,
            dx.data_ptr(), lddx, code, zero_tail)
    if out is not None:
        _written(out)
    return dx


def grouped_gemm_dw(dy, x, counts, out=None, out_dtype=None):
    """Gradient of grouped_gemm's weights: dW[e] = sum over expert e's rows of
    dy[r]^T x[r]. Returns dw [E, N, K]; an expert without rows gets zeros."""
    index = dy.get_device()
    if (index < 0 or dy.dtype is not _BF16 or dy.dim() != 2 or x.dtype is not _BF16 or x.dim() != 2
            or counts.dtype is not _I32 or counts.dim() != 1 or x.get_device() != index or counts.get_device() != index
            or not counts.is_contiguous()):
        _refuse("grouped_gemm_dw", _DW, dy, x, counts)
    rows, N = dy.shape
    rows_x, K = x.shape
    if rows_x != rows:
        _refuse("grouped_gemm_dw", _DW, dy, x, counts)
    E = counts.numel()
    if (E | rows | N | K) > _MAX:
        _too_large("grouped_gemm_dw", E, rows, N, K)
    dw, _, code = _out("grouped_gemm_dw", out, out_dtype, dy, (E, N, K))
    lddy = N if dy.is_contiguous() else _pitch(dy, rows, N, "dy", "grouped_gemm_dw")
    ldx = K if x.is_contiguous() else _pitch(x, rows, K, "x", "grouped_gemm_dw")
    _launch("latentmoe_grouped_gemm_dw", index, dy.data_ptr(), lddy, x.data_ptr(), ldx, counts.data_ptr(), E, rows,
            N, K, dw.data_ptr(), code)
    if out is not None:
        _written(out)
    return dw


def quantize_fp8(x, block_rows=1):
    """e4m3 codes and fp32 scales of x, bf16 or fp32: [R, K] or [n_mat, R, K] with one
    scale per block_rows x 128 elements. block_rows 1 (activations): scales
    [..., R, ceil(K/128)]; 128 (weights): scales [..., ceil(R/128), ceil(K/128)]."""
    index = x.get_device()
    dims = x.dim()
    code = _CODE.get(x.dtype)
    if (block_rows != 1 and block_rows != 128) or code is None or index < 0 or (
            dims != 2 and (dims != 3 or not x.is_contiguous())):
        _refuse("quantize_fp8", _QUANT, x, block_rows)
    if dims == 2:
        R, K = x.shape
        n_mat, ldx = 1, K if x.is_contiguous() else _pitch(x, R, K, "x", "quantize_fp8")
        scales = x.new_empty(-(-R // block_rows), -(-K // 128), dtype=_F32)
    else:
        n_mat, R, K = x.shape
        ldx = K
        scales = x.new_empty(n_mat, -(-R // block_rows), -(-K // 128), dtype=_F32)
    if (n_mat | R | K) > _MAX:
        _too_large("quantize_fp8", n_mat, R, K)
    codes = x.new_empty(R, K, dtype=_F8) if dims == 2 else x.new_empty(n_mat, R, K, dtype=_F8)
    _launch("latentmoe_quantize_fp8", index, x.data_ptr(), ldx, code, n_mat, R, K, block_rows, codes.data_ptr(),
            scales.data_ptr())
    return codes, scales


def gemm_fp8(xq, xs, wq, ws, counts=None, out=None, out_dtype=None, zero_tail=False):
    """y[r, n] = sum over 128-blocks b of xs[r, b] ws[n / 128, b] (xq[r, b] . wq[n, b]),
    with quantize_fp8's codes and scales: xq [rows, K], xs [rows, ceil(K/128)]. Without
    counts wq is [N, K] and ws [ceil(N/128), ceil(K/128)]; with counts [E] int32 the rows
    are in expert order, wq is [E, N, K] and ws [E, ceil(N/128), ceil(K/128)]."""
    index = xq.get_device()
    dims = 2 if counts is None else 3
    wanted = _DENSE8 if counts is None else _GROUPED8
    if (index < 0 or xq.dtype is not _F8 or xq.dim() != 2 or xs.dtype is not _F32 or wq.dtype is not _F8 or wq.dim() != dims
            or ws.dtype is not _F32 or xs.get_device() != index or wq.get_device() != index or ws.get_device() != index
            or not (xq.is_contiguous() and xs.is_contiguous() and wq.is_contiguous() and ws.is_contiguous())):
        _refuse("gemm_fp8", wanted, xq, xs, wq, ws, counts)
    rows, K = xq.shape
    kb = -(-K // 128)
    if counts is None:
        E, ptr = 1, None
        N, Kw = wq.shape
        fit = ws.shape == (-(-N // 128), kb)
    else:
        E, N, Kw = wq.shape
        fit = (ws.shape == (E, -(-N // 128), kb) and counts.dtype is _I32 and counts.dim() == 1 and counts.numel() == E
               and counts.get_device() == index and counts.is_contiguous())
        ptr = counts.data_ptr()
    if not fit or Kw != K or xs.shape != (rows, kb):
        _refuse("gemm_fp8", wanted, xq, xs, wq, ws, counts)
    if (E | rows | N | K) > _MAX:
        _too_large("gemm_fp8", E, rows, N, K)
    y, ldy, code = _out("gemm_fp8", out, out_dtype, xq, (rows, N))
    _launch("latentmoe_gemm_fp8", index, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), ptr, E, rows, N, K,
            y.data_ptr(), ldy, code, zero_tail)
    if out is not None:
        _written(out)
    return y
