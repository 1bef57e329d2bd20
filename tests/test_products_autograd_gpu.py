"""grouped_gemm as part of an autograd graph: gradients against fp64 and differences, what is refused, streams and
graph capture.

Tolerance: the products' own (test_grouped_gpu.py). A gradient that arrives in fp32 is rounded to bf16 once before
the products: half a step, 2^-8, of every term."""
import pytest
import torch

import latentmoe_layer_b200 as lm
from test_grouped_gpu import check_dw, check_dx, make

pytestmark = pytest.mark.gpu
COUNTS, N, K = [37, 0, 90, 2], 136, 200


def leaves(rows=None, seed=0):
    x, dy, w, c = make(COUNTS, N, K, rows=rows, seed=seed)
    return x.requires_grad_(), dy, w.requires_grad_(), c


def test_gradients_reach_rows_and_weights():
    x, dy, w, c = leaves()
    y = lm.grouped_gemm(x, w, c)
    assert y.requires_grad and y.dtype == torch.bfloat16
    y.backward(dy)
    assert x.grad.dtype == w.grad.dtype == torch.bfloat16
    check_dx(x.grad, dy, w.detach(), COUNTS)
    check_dw(w.grad, dy, x.detach(), COUNTS)
    # the same bits as the calls give
    assert torch.equal(x.grad, lm.grouped_gemm_dx(dy, w.detach(), c)) and torch.equal(w.grad, lm.grouped_gemm_dw(dy, x.detach(), c))
    with torch.no_grad():
        assert torch.equal(y, lm.grouped_gemm(x, w, c))
        assert not lm.grouped_gemm(x, w, c).requires_grad


@pytest.mark.parametrize("which", ["x", "w"])
def test_one_leaf_alone(which):
    x, dy, w, c = leaves()
    (w if which == "x" else x).requires_grad_(False)
    lm.grouped_gemm(x, w, c).backward(dy)
    if which == "x":
        check_dx(x.grad, dy, w, COUNTS)
        assert w.grad is None
    else:
        check_dw(w.grad, dy, x, COUNTS)
        assert x.grad is None


def test_fp32_output_and_a_broadcast_gradient():
    """sum() hands down a gradient of stride 0; an fp32 output's gradient is fp32."""
    x, _, w, c = leaves()
    y = lm.grouped_gemm(x, w, c, out_dtype=torch.float32)
    y.sum().backward()
    ones = torch.ones(y.shape, device="cuda").bfloat16()
    check_dx(x.grad, ones, w.detach(), COUNTS)
    check_dw(w.grad, ones, x.detach(), COUNTS)
    x.grad = w.grad = None
    g = torch.randn(y.shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    lm.grouped_gemm(x, w, c, out_dtype=torch.float32).backward(g)
    at = 0
    for e, n in enumerate(COUNTS):
        gd, xd, wd = g[at:at + n].double(), x.detach()[at:at + n].double(), w.detach()[e].double()
        for got, ref, mag, terms in ((x.grad[at:at + n], gd @ wd, gd.abs() @ wd.abs(), N),
                                     (w.grad[e], gd.t() @ xd, gd.abs().t() @ xd.abs(), n)):
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 1.01 * (terms + 1) * 2.0 ** -23) * (1 + 2.0 ** -8) * mag + 1e-38
            assert ((got.double() - ref).abs() <= tol).all()
        at += n


def test_gradient_against_differences():
    x, dy, w, c = leaves(seed=4)
    (lm.grouped_gemm(x, w, c, out_dtype=torch.float32) * dy.float()).sum().backward()

    def loss(x, w):
        with torch.no_grad():
            return float((lm.grouped_gemm(x, w, c, out_dtype=torch.float32).double() * dy.double()).sum())

    base = loss(x, w)
    for r, k, e, n in ((0, 3, 0, 5), (40, 199, 2, 135), (128, 0, 3, 0), (126, 77, 2, 64)):
        x2, w2 = x.detach().clone(), w.detach().clone()
        x2[r, k] += 2.0
        w2[e, n, k] += 2.0
        # the product is linear: fp32 y (200 * 2^-23 of |x||w| <= 200 * 25 each, times |dy| <= 5 and at most 136
        # elements) gives the quotient 0.05; the gradient's rounding to bf16 is 2^-8 of it
        for got, q in ((x.grad[r, k], (loss(x2, w) - base) / float(x2[r, k].double() - x.detach()[r, k].double())),
                       (w.grad[e, n, k], (loss(x, w2) - base) / float(w2[e, n, k].double() - w.detach()[e, n, k].double()))):
            assert abs(float(got) - q) <= 0.05 + 2.0 ** -8 * abs(q)


def test_padded_batch():
    """Rows behind the last group: neither their outputs' gradients nor what they hold reach a gradient."""
    x, dy, w, c = leaves(rows=150)
    with torch.no_grad():
        x[129:] = float("nan")
        dy[129:] = float("nan")
    lm.grouped_gemm(x, w, c).backward(dy)
    check_dx(x.grad, dy, w.detach(), COUNTS)
    check_dw(w.grad, dy, x.detach(), COUNTS)
    assert not x.grad[129:].any()


def test_few_rows_none_and_strided_rows():
    wide = torch.randn(3, 264, device="cuda").bfloat16().requires_grad_()
    _, _, w, _ = leaves()
    c = torch.tensor([2, 0, 1, 0], dtype=torch.int32, device="cuda")
    y = lm.grouped_gemm(wide[:, 16:216], w, c)
    dy = torch.randn_like(y)
    y.backward(dy)
    check_dx(wide.grad[:, 16:216], dy, w.detach(), [2, 0, 1, 0])
    check_dw(w.grad, dy, wide.detach()[:, 16:216], [2, 0, 1, 0])
    assert not wide.grad[:, :16].any() and not wide.grad[:, 216:].any()
    w.grad = None
    none = torch.empty(0, K, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    lm.grouped_gemm(none, w, torch.zeros(4, dtype=torch.int32, device="cuda")).sum().backward()
    assert none.grad.shape == (0, K) and not w.grad.any()


def test_what_is_refused():
    x, dy, w, c = leaves()
    with pytest.raises(ValueError):  # as torch's own functions with out=
        lm.grouped_gemm(x, w, c, out=torch.empty(129, N, dtype=torch.bfloat16, device="cuda"))
    with torch.no_grad():
        lm.grouped_gemm(x, w, c, out=torch.empty(129, N, dtype=torch.bfloat16, device="cuda"))
    g, = torch.autograd.grad(lm.grouped_gemm(x, w, c).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        g.float().sum().backward()
    y = lm.grouped_gemm(x, w, c)
    c += 1
    with pytest.raises(RuntimeError):  # the counts that the backward pass would read have changed
        y.backward(dy)


@pytest.mark.parametrize("call", ["forward", "dx", "dw", "fp8"])
def test_writing_to_out_is_seen_by_autograd(call):
    x, dy, w, c = make(COUNTS, N, K)
    xq, xs = lm.quantize_fp8(torch.randn(129, 208, device="cuda"))
    wq, ws = lm.quantize_fp8(torch.randn(4, N, 208, device="cuda"), block_rows=128)
    run, shape = {"forward": (lambda o: lm.grouped_gemm(x, w, c, out=o), (129, N)),
                  "dx": (lambda o: lm.grouped_gemm_dx(dy, w, c, out=o), (129, K)),
                  "dw": (lambda o: lm.grouped_gemm_dw(dy, x, c, out=o), (4, N, K)),
                  "fp8": (lambda o: lm.gemm_fp8(xq, xs, wq, ws, counts=c, out=o), (129, N))}[call]
    out = torch.ones(shape, device="cuda")
    leaf = torch.ones(shape, device="cuda", requires_grad=True)
    loss = (leaf * out).sum()  # its backward pass needs out as it is now
    run(out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        run(torch.ones(shape, device="cuda"))


def step(x, up, down, c):
    h = lm.grouped_gemm(x, up, c, zero_tail=True)
    y = lm.grouped_gemm(torch.relu(h).square(), down, c, zero_tail=True)
    return (y.float() ** 2).sum()


def test_on_a_side_stream_and_captured():
    """A training step's gradients are the same bits on another stream, and replayed from a graph while an
    eager graph of other leaves lives."""
    x, _, up, c = leaves()
    down = (torch.randn(4, K, N, device="cuda") * 0.1).bfloat16().requires_grad_()
    step(x, up, down, c).backward()
    want = [t.grad.clone() for t in (x, up, down)]

    def again():
        return [t.detach().clone().requires_grad_() for t in (x, up, down)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = again()
        step(*a, c).backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(t.grad, g) for t, g in zip(a, want))
    eager = step(*again(), c)
    b = again()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up on the capture's kind of stream
        step(*b, c).backward()
    torch.cuda.current_stream().wait_stream(side)
    for t in b:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*b, c).backward()
    for _ in range(3):
        for t in b:
            t.grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t.grad, g) for t, g in zip(b, want))
    eager.backward()
