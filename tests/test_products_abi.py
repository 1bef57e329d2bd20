"""Refusals of the products without a handle: every bad argument gives its status before any CUDA call,
so these run without a GPU (the addresses are made up and never touched)."""
import ctypes

import pytest

import latentmoe_layer_b200 as lm

A = 0x10000  # an aligned address
OK, INVALID, UNSUPPORTED = lm.LMOE_OK, lm.LMOE_ERR_INVALID_ARG, lm.LMOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from latentmoe_layer_b200 import build
    build.build()
    return lm.load()


def grouped(fn, **kw):
    """x (or dy), w, counts, sizes and output, all valid unless replaced."""
    a = dict(x=A, ldx=None, w=A, counts=A, E=4, rows=64, N=136, K=72, y=A, ldy=None, dtype=0)
    a.update(kw)
    dx = fn == "latentmoe_grouped_gemm_dx"
    if a["ldx"] is None:
        a["ldx"] = a["N"] if dx else a["K"]
    if a["ldy"] is None:
        a["ldy"] = a["K"] if dx else a["N"]
    return getattr(lm.load(), fn)(a["x"], a["ldx"], a["w"], a["counts"], a["E"], a["rows"], a["N"], a["K"], a["y"], a["ldy"],
                                  a["dtype"], 0, None)


@pytest.mark.parametrize("fn", ["latentmoe_grouped_gemm", "latentmoe_grouped_gemm_dx"])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=0, x=None, y=None), OK),            # nothing to do
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(counts=None), INVALID), (dict(y=None), INVALID),
    (dict(x=A + 2), INVALID), (dict(w=A + 8), INVALID), (dict(counts=A + 2), INVALID), (dict(y=A + 4), INVALID),
    (dict(ldx=64), INVALID), (dict(ldx=147), INVALID), (dict(ldy=64), INVALID), (dict(ldy=148), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(N=100), UNSUPPORTED), (dict(K=20), UNSUPPORTED), (dict(N=1 << 23), UNSUPPORTED),
    (dict(K=1 << 23), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(E=1024, N=1 << 20, K=1 << 12), UNSUPPORTED), (dict(rows=1 << 30, ldx=1 << 20), UNSUPPORTED),
    (dict(rows=1 << 30, N=1 << 22, ldx=1 << 22, ldy=1 << 22), UNSUPPORTED),
])
def test_grouped_refusals(lib, fn, kw, status):
    assert grouped(fn, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(dy=None), INVALID), (dict(x=None), INVALID),
    (dict(counts=None), INVALID), (dict(dw=None), INVALID), (dict(dw=A + 8), INVALID), (dict(lddy=128), INVALID),
    (dict(ldx=76), INVALID), (dict(dtype=7), INVALID), (dict(N=12), UNSUPPORTED), (dict(K=4), UNSUPPORTED),
    (dict(E=2000), UNSUPPORTED), (dict(E=1024, N=1 << 22, K=1 << 22), UNSUPPORTED),
])
def test_weight_gradient_refusals(lib, kw, status):
    a = dict(dy=A, lddy=136, x=A, ldx=72, counts=A, E=4, rows=64, N=136, K=72, dw=A, dtype=1)
    a.update(kw)
    assert lib.latentmoe_grouped_gemm_dw(a["dy"], a["lddy"], a["x"], a["ldx"], a["counts"], a["E"], a["rows"], a["N"], a["K"],
                                         a["dw"], a["dtype"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_mat=0), OK), (dict(R=0, x=None, codes=None, scales=None), OK),
    (dict(n_mat=-1), INVALID), (dict(R=-1), INVALID), (dict(K=0), INVALID), (dict(block=64), INVALID), (dict(dtype=3), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=A + 2), INVALID),
    (dict(codes=A + 8), INVALID), (dict(scales=A + 2), INVALID), (dict(ldx=128), INVALID), (dict(ldx=260), INVALID),
    (dict(K=264, ldx=264), UNSUPPORTED), (dict(n_mat=65536), UNSUPPORTED), (dict(K=1 << 23, ldx=1 << 23), UNSUPPORTED),
    (dict(n_mat=65535, R=1 << 20), UNSUPPORTED), (dict(R=65536 * 128, block=128), UNSUPPORTED),
    (dict(R=2 ** 31 - 15, K=16, ldx=16), UNSUPPORTED),  # the last CTA's rows would pass 32 bits
])
def test_quantiser_refusals(lib, kw, status):
    a = dict(x=A, ldx=256, dtype=0, n_mat=1, R=64, K=256, block=1, codes=A, scales=A)
    a.update(kw)
    assert lib.latentmoe_quantize_fp8(a["x"], a["ldx"], a["dtype"], a["n_mat"], a["R"], a["K"], a["block"], a["codes"],
                                      a["scales"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0, xq=None, xs=None, y=None), OK), (dict(counts=None), INVALID),  # one matrix only without counts
    (dict(counts=None, E=1, rows=0), OK), (dict(counts=A + 1), INVALID), (dict(xq=None), INVALID), (dict(xs=None), INVALID),
    (dict(wq=None), INVALID), (dict(ws=None), INVALID), (dict(xs=A + 4), INVALID), (dict(ws=A + 8), INVALID),
    (dict(wq=A + 8), INVALID), (dict(y=None), INVALID), (dict(ldy=128), INVALID), (dict(ldy=140), INVALID),
    (dict(dtype=2), INVALID), (dict(K=72), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
])
def test_8_bit_product_refusals(lib, kw, status):
    a = dict(xq=A, xs=A, wq=A, ws=A, counts=A, E=4, rows=64, N=136, K=272, y=A, ldy=136, dtype=0)
    a.update(kw)
    assert lib.latentmoe_gemm_fp8(a["xq"], a["xs"], a["wq"], a["ws"], a["counts"], a["E"], a["rows"], a["N"], a["K"], a["y"],
                                  a["ldy"], a["dtype"], 0, None) == status


def test_binding_refuses_cpu_tensors_and_importing_it_does_not_import_torch():
    import subprocess
    import sys
    import torch
    x, w, c = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 8, 16).bfloat16(), torch.zeros(2, dtype=torch.int32)
    f8 = torch.zeros(4, 16).to(torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    for call in (lambda: lm.grouped_gemm(x, w, c), lambda: lm.grouped_gemm_dx(x, w, c), lambda: lm.grouped_gemm_dw(x, x, c),
                 lambda: lm.quantize_fp8(x), lambda: lm.gemm_fp8(f8, s, f8, s)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        lm.no_such_product
    code = "import sys, latentmoe_layer_b200; sys.exit('torch' in sys.modules)"
    assert subprocess.run([sys.executable, "-c", code], cwd=__file__.rsplit("/tests/", 1)[0]).returncode == 0


def test_status_and_wait_limit_without_a_gpu(lib):
    assert lm.latentmoe_products_status() == OK  # nothing has run
    for polls, status in ((-1, INVALID), (1 << 32, INVALID), (0, OK), ((1 << 32) - 1, OK), (1 << 24, OK)):
        assert lm.latentmoe_set_products_wait_limit(polls) == status
