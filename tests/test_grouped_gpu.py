"""Grouped expert products and their gradients against the definition in fp64.

Tolerance, derived: a sum of n products accumulated in fp32 with one rounding or
truncation per addition is off by at most n * 2^-23 * sum |a b| (n covers the
additions between chunks too); rounding the result is off by half a step, 2^-8
(bf16) or 2^-24 (fp32) of its value. Both terms are taken per element.
"""
import numpy as np
import pytest
import torch

import latentmoe_layer_b200 as lm
import synth

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def spread(total, groups, seed, empty=0.2):
    """Uneven counts that add up to total, some of them zero."""
    rng = np.random.default_rng(seed)
    p = rng.exponential(size=groups) * (rng.random(groups) >= empty)
    if p.sum() == 0:
        p[-1] = 1.0
    return rng.multinomial(total, p / p.sum()).tolist()


def make(counts, N, K, rows=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = sum(counts) if rows is None else rows
    E = len(counts)
    x = torch.randn(rows, K, generator=g, device="cuda").bfloat16()
    dy = torch.randn(rows, N, generator=g, device="cuda").bfloat16()
    w = torch.randn(E, N, K, generator=g, device="cuda").bfloat16()
    return x, dy, w, torch.tensor(counts, dtype=torch.int32, device="cuda")


def check(got, ref, mag, n):
    """got against ref (fp64) with mag = the same sum over absolute values."""
    assert torch.isfinite(got).all()
    d = (got.double() - ref).abs()
    tol = HALF_STEP[got.dtype] * ref.abs() + (1 + 2.0 ** -8) * n * 2.0 ** -23 * mag + 1e-38
    worst = float((d / tol).max()) if d.numel() else 0.0
    assert worst <= 1.0, worst


def check_forward(y, x, w, counts):
    at = 0
    for e, n in enumerate(counts):
        if n:
            a, b = x[at:at + n].double(), w[e].double()
            check(y[at:at + n], a @ b.t(), a.abs() @ b.abs().t(), w.shape[2] + 1)
        at += n


def check_dx(dx, dy, w, counts):
    at = 0
    for e, n in enumerate(counts):
        if n:
            a, b = dy[at:at + n].double(), w[e].double()
            check(dx[at:at + n], a @ b, a.abs() @ b.abs(), w.shape[1] + 1)
        at += n


def check_dw(dw, dy, x, counts):
    at = 0
    for e, n in enumerate(counts):
        a, b = dy[at:at + n].double(), x[at:at + n].double()
        check(dw[e], a.t() @ b, a.abs().t() @ b.abs(), n + 1)
        at += n


CASES = [
    # counts, N, K; up to 8 rows take another kernel than more
    ([1] + [0] * 500 + [3, 0, 1], 40, 1032), ([0, 8], 136, 2048), ([9], 136, 2048), ([1] * 8, 72, 520), ([4, 0, 5], 24, 72),
    ([5], 8, 8),
    ([1], 64, 64),
    ([0, 0, 3, 0], 128, 64),
    ([0, 0, 0, 7], 16, 24),
    ([31, 32, 33, 0, 1], 136, 72),
    ([64, 63, 65, 128], 264, 200),
    ([255, 256, 257], 256, 128),
    ([513, 0, 130, 700], 520, 1032),
    ([300], 2048, 2560),
    (spread(1031, 37, 1), 264, 456),
    (spread(40, 128, 2), 512, 512),
    (spread(333, 1024, 3, empty=0.7), 40, 48),
    ([2999, 0, 64 * 40, 64 * 13 + 1, 7, 1600 - 3], 1288, 776),  # many k-blocks between partial ones
    (spread(9000, 24, 4), 520, 264),
    # few tiles and a long contraction (for dx: N): shared by two or four pairs of SMs
    ([40], 264, 4096), ([20, 0, 30], 136, 2952), ([200], 520, 2056), ([100, 28], 4104, 72), ([0, 300], 2568, 520), ([90], 72, 456),
]
IDS = ["%dx%d e%d r%d" % (n, k, len(c), sum(c)) for c, n, k in CASES]


@pytest.mark.parametrize("counts,N,K", CASES, ids=IDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_forward(counts, N, K, dtype):
    x, _, w, c = make(counts, N, K)
    y = lm.grouped_gemm(x, w, c, out_dtype=dtype)
    assert y.dtype == dtype and y.shape == (sum(counts), N)
    check_forward(y, x, w, counts)


@pytest.mark.parametrize("counts,N,K", CASES, ids=IDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_input_gradient(counts, N, K, dtype):
    _, dy, w, c = make(counts, N, K)
    dx = lm.grouped_gemm_dx(dy, w, c, out_dtype=dtype)
    assert dx.dtype == dtype and dx.shape == (sum(counts), K)
    check_dx(dx, dy, w, counts)


@pytest.mark.parametrize("counts,N,K", CASES, ids=IDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_weight_gradient(counts, N, K, dtype):
    x, dy, _, c = make(counts, N, K)
    dw = lm.grouped_gemm_dw(dy, x, c, out_dtype=dtype)
    assert dw.dtype == dtype and dw.shape == (len(counts), N, K)
    check_dw(dw, dy, x, counts)
    for e, n in enumerate(counts):
        if n == 0:
            assert not dw[e].any()


def test_gradients_against_differences():
    """The product is linear, so a difference quotient of sum(dy * y) has no error of its own."""
    counts, N, K = [3, 0, 40, 21], 24, 40
    x, dy, w, c = make(counts, N, K, seed=4)
    dx = lm.grouped_gemm_dx(dy, w, c, out_dtype=torch.float32)
    dw = lm.grouped_gemm_dw(dy, x, c, out_dtype=torch.float32)

    def loss(x, w):
        return float((lm.grouped_gemm(x, w, c, out_dtype=torch.float32).double() * dy.double()).sum())

    base = loss(x, w)
    g = torch.Generator().manual_seed(1)
    for _ in range(12):
        r, k = int(torch.randint(64, (), generator=g)), int(torch.randint(K, (), generator=g))
        n, e = int(torch.randint(N, (), generator=g)), int(torch.tensor([0, 2, 3])[torch.randint(3, (), generator=g)])
        x2, w2 = x.clone(), w.clone()
        x2[r, k] += 2.0
        w2[e, n, k] += 2.0
        # fp32 y: K * 2^-23 * |x||w| per element, at most 40 * 2^-23 * 40 * 25, times |dy| and N or the rows: below 0.05
        assert abs((loss(x2, w) - base) / float(x2[r, k].double() - x[r, k].double()) - float(dx[r, k])) < 0.05
        assert abs((loss(x, w2) - base) / float(w2[e, n, k].double() - w[e, n, k].double()) - float(dw[e, n, k])) < 0.05


@pytest.mark.parametrize("zero_tail", [False, True])
def test_rows_behind_the_last_group(zero_tail):
    """Rows behind the last group may hold NaN: nobody reads them, and their outputs stay or become zero."""
    check_tail([40, 0, 300, 17], 700, 136, 264, zero_tail)
    check_tail([20, 0, 9], 60, 2568, 2056, zero_tail)  # contraction shared by four pairs
    check_tail([0, 0], 40, 136, 2056, zero_tail)


def check_tail(counts, rows, N, K, zero_tail):
    x, dy, w, c = make(counts, N, K, rows=rows)
    used = sum(counts)
    x[used:] = float("nan")
    dy[used:] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.full((rows, N), -7.0, dtype=dtype, device="cuda")
        dx = torch.full((rows, K), -7.0, dtype=dtype, device="cuda")
        assert lm.grouped_gemm(x, w, c, out=y, zero_tail=zero_tail) is y
        lm.grouped_gemm_dx(dy, w, c, out=dx, zero_tail=zero_tail)
        dw = lm.grouped_gemm_dw(dy, x, c, out_dtype=dtype)
        check_forward(y, x, w, counts)
        check_dx(dx, dy, w, counts)
        check_dw(dw, dy, x, counts)
        left = 0.0 if zero_tail else -7.0
        assert (y[used:] == left).all() and (dx[used:] == left).all()


@pytest.mark.parametrize("counts,rows", [([0, 1, 0], 8), ([0, 0], 5), ([2, 0, 3], 8), ([1], 1), ([3], 7)])
def test_few_rows_and_a_tail(counts, rows):
    N, K = 136, 264
    x, dy, w, c = make(counts, N, K, rows=rows)
    used = sum(counts)
    x[used:] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        for zero_tail in (False, True):
            y = torch.full((rows, N), -7.0, dtype=dtype, device="cuda")
            lm.grouped_gemm(x, w, c, out=y, zero_tail=zero_tail)
            check_forward(y, x, w, counts)
            assert (y[used:] == (0.0 if zero_tail else -7.0)).all()
    for over in ([5, 1 << 30, 7], [-1, 2, 1 << 30]):
        c3 = torch.tensor(over, dtype=torch.int32, device="cuda")
        w3 = torch.randn(3, N, K, device="cuda").bfloat16()
        x3 = torch.randn(rows, K, device="cuda").bfloat16()
        first = max(0, min(over[0], rows))
        second = max(0, min(over[1], rows - first))
        check_forward(lm.grouped_gemm(x3, w3, c3), x3, w3, [first, second, rows - first - second])


# CTAs of 16 columns and a group with rows: 148 SMs hold 444 of eight warps and 888 of four
LARGE_GRIDS = [([1], 8200, 24), ([8], 8200, 1032), ([5], 14216, 520), ([2, 0, 3, 1], 2408, 2056), ([0, 1, 7], 5000, 72),
               ([1, 2, 1, 1, 1, 1], 2456, 136), ([0, 1, 1, 2, 1, 1, 2], 2568, 712), ([3], 7112, 64), ([3], 14200, 200)]


@pytest.mark.parametrize("counts,N,K", LARGE_GRIDS, ids=["%dx%d e%d r%d" % (n, k, len(c), sum(c)) for c, n, k in LARGE_GRIDS])
@pytest.mark.parametrize("tail", [0, 2])
def test_few_rows_on_large_grids(counts, N, K, tail):
    rows = min(8, sum(counts) + tail)
    x, _, w, c = make(counts, N, K, rows=rows)
    used = sum(counts)
    x[used:] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        for zero_tail in (False, True):
            y = torch.full((rows, N), -7.0, dtype=dtype, device="cuda")
            lm.grouped_gemm(x, w, c, out=y, zero_tail=zero_tail)
            check_forward(y, x, w, counts)
            assert (y[used:] == (0.0 if zero_tail else -7.0)).all()


def test_counts_that_do_not_fit():
    """Negative counts are empty groups; rows past the batch do not exist."""
    N, K = 72, 136
    x, dy, w, _ = make([100, 0, 80, 60], N, K)
    c = torch.tensor([100, -5, 80, 1 << 30], dtype=torch.int32, device="cuda")
    counts = [100, 0, 80, 60]
    check_forward(lm.grouped_gemm(x, w, c), x, w, counts)
    check_dx(lm.grouped_gemm_dx(dy, w, c), dy, w, counts)
    check_dw(lm.grouped_gemm_dw(dy, x, c), dy, x, counts)
    big = torch.full((4,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    check_forward(lm.grouped_gemm(x, w, big), x, w, [240, 0, 0, 0])
    check_dw(lm.grouped_gemm_dw(dy, x, big), dy, x, [240, 0, 0, 0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_group(bad):
    counts, N, K = [70, 33, 100], 136, 72
    x, dy, w, c = make(counts, N, K)
    x[70:103] = bad
    dy[70:103] = bad
    y = lm.grouped_gemm(x, w, c)
    dx = lm.grouped_gemm_dx(dy, w, c)
    dw = lm.grouped_gemm_dw(dy, x, c)
    keep = torch.ones(203, dtype=torch.bool, device="cuda")
    keep[70:103] = False
    for e, (lo, hi) in enumerate([(0, 70), (70, 103), (103, 203)]):
        if e == 1:
            assert not torch.isfinite(y[lo:hi]).any() and not torch.isfinite(dx[lo:hi]).any()
            assert not torch.isfinite(dw[e]).any()
            continue
        check_forward(y[lo:hi], x[lo:hi], w[e:e + 1], [hi - lo])
        check_dx(dx[lo:hi], dy[lo:hi], w[e:e + 1], [hi - lo])
        check_dw(dw[e:e + 1], dy[lo:hi], x[lo:hi], [hi - lo])


def test_row_pitch():
    """Inputs and outputs that are column ranges of wider tensors."""
    counts, N, K = [37, 90, 2], 136, 200
    x, dy, w, c = make(counts, N, K)
    wide_x = torch.full((129, K + 48), float("nan"), device="cuda").bfloat16()
    wide_dy = torch.full((129, N + 16), float("nan"), device="cuda").bfloat16()
    wide_x[:, 16:16 + K] = x
    wide_dy[:, 8:8 + N] = dy
    xs, dys = wide_x[:, 16:16 + K], wide_dy[:, 8:8 + N]
    wide_y = torch.full((129, N + 24), 5.0, device="cuda").bfloat16()
    y = lm.grouped_gemm(xs, w, c, out=wide_y[:, 8:8 + N])
    check_forward(y, x, w, counts)
    assert (wide_y[:, :8] == 5).all() and (wide_y[:, 8 + N:] == 5).all()
    check_dx(lm.grouped_gemm_dx(dys, w, c), dy, w, counts)
    check_dw(lm.grouped_gemm_dw(dys, xs, c), dy, x, counts)
    # one row of a wider tensor, at an offset
    one = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    check_forward(lm.grouped_gemm(xs[40:41], w, one), x[40:41], w, [0, 1, 0])


def test_no_rows():
    w = torch.randn(3, 64, 128, device="cuda").bfloat16()
    c = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert lm.grouped_gemm(x, w, c).shape == (0, 64)
    assert lm.grouped_gemm_dx(dy, w, c).shape == (0, 128)
    out = torch.full((3, 64, 128), 3.0, device="cuda")
    assert not lm.grouped_gemm_dw(dy, x, c, out=out).any()


def test_same_bits_again_and_on_another_stream():
    counts = spread(2000, 19, 7)
    x, dy, w, c = make(counts, 520, 1032)
    first = (lm.grouped_gemm(x, w, c), lm.grouped_gemm_dx(dy, w, c), lm.grouped_gemm_dw(dy, x, c, out_dtype=torch.float32))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # both streams' calls are in flight at once
        with torch.cuda.stream(s):
            got.append((lm.grouped_gemm(x, w, c), lm.grouped_gemm_dx(dy, w, c),
                        lm.grouped_gemm_dw(dy, x, c, out_dtype=torch.float32)))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(first, g):
            assert torch.equal(a, b)


def test_graph_replays_with_other_counts():
    """A captured call reads the counts and the rows at replay."""
    x, dy, w, c = make([200, 100, 0, 156], 264, 200)
    y, dx = torch.empty(456, 264, device="cuda").bfloat16(), torch.empty(456, 200, device="cuda").bfloat16()
    dw = torch.empty(4, 264, 200, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.grouped_gemm(x, w, c, out=y)
        lm.grouped_gemm_dx(dy, w, c, out=dx)
        lm.grouped_gemm_dw(dy, x, c, out=dw)
    for counts in ([200, 100, 0, 156], [1, 0, 455, 0], [114, 114, 114, 114]):
        c.copy_(torch.tensor(counts, dtype=torch.int32))
        x.copy_(torch.randn_like(x, dtype=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        check_forward(y, x, w, counts)
        check_dx(dx, dy, w, counts)
        check_dw(dw, dy, x, counts)


SHAPE = synth.LayerShape("products", T=97, H=256, L=128, E=16, k=4, G=4, Gk=2, I=320, Is=256)


def test_expert_stage_from_the_products():
    """Rows and counts of latentmoe_ep_front through the products give the layer's expert stage:
    o = w * down(relu2(up(row)))."""
    dev = synth.device_inputs(SHAPE, 0)
    layer = lm.LatentMoE(SHAPE, dev, SHAPE.T)
    A = SHAPE.T * SHAPE.k
    rows = torch.empty((A, SHAPE.L), dtype=torch.bfloat16, device="cuda")
    rw = torch.empty((A,), dtype=torch.float32, device="cuda")
    counts = torch.empty((SHAPE.E,), dtype=torch.int32, device="cuda")
    layer.ep_front(dev["x"], rows, rw, counts)
    o = torch.empty((A, SHAPE.L), dtype=torch.float32, device="cuda")
    layer.ep_experts(rows, rw, counts, 1, o)
    up, down = dev["up_w"].view(SHAPE.E, SHAPE.I, SHAPE.L), dev["down_w"].view(SHAPE.E, SHAPE.L, SHAPE.I)
    h = lm.grouped_gemm(rows, up, counts, out_dtype=torch.float32)
    a = torch.relu(h).square().bfloat16()
    mine = lm.grouped_gemm(a, down, counts, out_dtype=torch.float32) * rw[:, None]
    # a differs from the layer's by single bf16 roundings of the activations (2^-8 of |a| each, where the
    # two fp32 sums straddle a rounding border): |a| |down| * 2^-8 bounds what each can move
    at = 0
    for e, n in enumerate(counts.tolist()):
        if n:
            sl = slice(at, at + n)
            mag = a[sl].double() @ down[e].double().abs().t() * rw[sl, None].double()
            assert ((mine[sl] - o[sl]).double().abs() <= 2.0 ** -8 * mag + 1e-30).all()
        at += n
    layer.close()


class ExpertProduct(torch.autograd.Function):
    """How a training program uses the three calls."""

    @staticmethod
    def forward(ctx, x, w, counts):
        ctx.save_for_backward(x, w, counts)
        return lm.grouped_gemm(x, w, counts, zero_tail=True)

    @staticmethod
    def backward(ctx, dy):
        x, w, counts = ctx.saved_tensors
        dy = dy.contiguous()
        return lm.grouped_gemm_dx(dy, w, counts, zero_tail=True), lm.grouped_gemm_dw(dy, x, counts), None


def test_expert_layer_trains():
    """up, relu2, down and back on a padded batch: gradients of both weights and of the rows against fp64."""
    counts, rows, L, I = [30, 0, 65, 9], 128, 64, 96
    used = sum(counts)
    x, _, _, c = make(counts, I, L, rows=rows)
    g = torch.Generator(device="cuda").manual_seed(9)
    up = (torch.randn(4, I, L, generator=g, device="cuda") * 0.1).bfloat16().requires_grad_()
    down = (torch.randn(4, L, I, generator=g, device="cuda") * 0.1).bfloat16().requires_grad_()
    x.requires_grad_()
    h = ExpertProduct.apply(x, up, c)
    y = ExpertProduct.apply(torch.relu(h).square(), down, c)
    (y[:used].float() ** 2).sum().backward()
    ux, uu, ud = [t.detach().double().requires_grad_() for t in (x, up, down)]
    outs, at = [], 0
    for e, n in enumerate(counts):
        outs.append(torch.relu(ux[at:at + n] @ uu[e].t()).square() @ ud[e].t())
        at += n
    (torch.cat(outs) ** 2).sum().backward()
    # every tensor of the chain (h, a, y, dy, da, dh and the gradient) is rounded to bf16 once: seven
    # roundings of 2^-8, the square doubles h's two (in a and in da), and each enters the gradient's
    # norm at most linearly through sums of like-sized terms: 10 * 2^-8
    for got, ref in ((x.grad, ux.grad), (up.grad, uu.grad), (down.grad, ud.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) < 10 * 2.0 ** -8
    assert not x.grad[used:].any() and not up.grad[1].any() and not down.grad[1].any()


def test_refusals_of_the_binding():
    x, dy, w, c = make([3, 5], 24, 40)
    bad = [lambda: lm.grouped_gemm(x.float(), w, c), lambda: lm.grouped_gemm(x, w[0], c), lambda: lm.grouped_gemm(x, w, c.long()),
           lambda: lm.grouped_gemm(x, w, c[:1]), lambda: lm.grouped_gemm(x, w.transpose(1, 2), c),
           lambda: lm.grouped_gemm(x, w, c.cpu()), lambda: lm.grouped_gemm(x.cpu(), w, c), lambda: lm.grouped_gemm(dy, w, c),
           lambda: lm.grouped_gemm(x.t(), w, c), lambda: lm.grouped_gemm(x[:1].expand(8, 40), w, c),
           lambda: lm.grouped_gemm(x, w, c, out=torch.empty(8, 24, device="cuda").half()),
           lambda: lm.grouped_gemm(x, w, c, out=torch.empty(7, 24, device="cuda")),
           lambda: lm.grouped_gemm(x, w, c, out=torch.empty(24, 8, device="cuda").t()),
           lambda: lm.grouped_gemm(x, w, c, out=torch.empty(8, 24, device="cuda"), out_dtype=torch.bfloat16),
           lambda: lm.grouped_gemm(x, w, c, out_dtype=torch.float16), lambda: lm.grouped_gemm_dx(x, w, c),
           lambda: lm.grouped_gemm_dw(dy, x[:4], c), lambda: lm.grouped_gemm_dw(dy, x, c.view(2, 1)),
           lambda: lm.grouped_gemm_dw(dy, x, c, out=torch.empty(2, 40, 24, device="cuda").transpose(1, 2))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(8, 48, device="cuda").bfloat16()
    w42 = torch.zeros(2, 24, 42, device="cuda").bfloat16()
    for call, status in ((lambda: lm.grouped_gemm(wide[:, 1:41], w, c), lm.LMOE_ERR_INVALID_ARG),  # rows not 16-byte aligned
                         (lambda: lm.grouped_gemm(torch.zeros(8, 42, device="cuda").bfloat16(), w42, c), lm.LMOE_ERR_UNSUPPORTED)):
        with pytest.raises(lm.LmoeError) as e:
            call()
        assert e.value.status == status


FIRST = """
import sys, torch
sys.path.insert(0, %r)
import latentmoe_layer_b200 as lm
x = torch.randn(40, 64, device="cuda").bfloat16()
w = torch.randn(2, 72, 64, device="cuda").bfloat16()
c = torch.tensor([15, 25], dtype=torch.int32, device="cuda")
y, dw = torch.zeros(40, 72, device="cuda"), torch.zeros(2, 72, 64, device="cuda")
dy = torch.randn(40, 72, device="cuda").bfloat16()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):   # the library's first calls in this process
    lm.grouped_gemm(x, w, c, out=y)
    lm.grouped_gemm_dw(dy, x, c, out=dw)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, lm.grouped_gemm(x, w, c, out_dtype=torch.float32)) and y.abs().sum() > 0
assert torch.equal(dw, lm.grouped_gemm_dw(dy, x, c, out_dtype=torch.float32)) and dw.abs().sum() > 0
print("captured first")
"""


def test_first_call_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % root], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout[-2000:]


def test_two_threads_at_once():
    """Calls from two host threads, each on a stream of its own."""
    import threading
    jobs = []
    for seed in range(2):
        counts = spread(700, 9, seed)
        x, dy, w, c = make(counts, 264, 520, seed=seed)
        jobs.append((counts, x, dy, w, c, torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def work(job):
        counts, x, dy, w, c, stream, got = job
        with torch.cuda.stream(stream):
            for _ in range(20):
                got.append((lm.grouped_gemm(x, w, c), lm.grouped_gemm_dw(dy, x, c, out_dtype=torch.float32)))

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for counts, x, dy, w, c, _, got in jobs:
        assert len(got) == 20
        check_forward(got[0][0], x, w, counts)
        check_dw(got[0][1], dy, x, counts)
        assert all(torch.equal(got[0][0], y) and torch.equal(got[0][1], dw) for y, dw in got)


def test_first_cuda_use_of_a_thread():
    """A thread that has made no CUDA call yet, nor torch for it."""
    import threading
    counts, N, K = [40, 0, 77], 136, 264
    x, dy, w, c = make(counts, N, K)
    y, dx, dw = lm.grouped_gemm(x, w, c), lm.grouped_gemm_dx(dy, w, c), lm.grouped_gemm_dw(dy, x, c)
    for run, out, want in ((lambda o: lm.grouped_gemm(x, w, c, out=o), torch.zeros_like(y), y),
                           (lambda o: lm.grouped_gemm_dx(dy, w, c, out=o), torch.zeros_like(dx), dx),
                           (lambda o: lm.grouped_gemm_dw(dy, x, c, out=o), torch.zeros_like(dw), dw)):
        torch.cuda.synchronize()
        failed = []

        def work():
            try:
                run(out)
            except Exception as e:
                failed.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not failed and torch.equal(out, want), failed


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_long_sums_of_one_sign(dtype):
    """Contractions of 2^22 like-signed products, where an error of every addition has the same sign.

    Tolerance: at most 4096 products are summed in the tensor core before the sum goes into an fp32
    register, one of the 1024 sums added there: (4096 + 1024) * 2^-23 of the sum, and rounding the result."""
    n = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(5)
    a = (torch.rand(n, 16, generator=g, device="cuda") + 0.5).bfloat16()
    b = (torch.rand(n, 24, generator=g, device="cuda") + 0.5).bfloat16()
    ref = torch.zeros(16, 24, dtype=torch.float64, device="cuda")
    for at in range(0, n, 1 << 18):
        ref += a[at:at + (1 << 18)].double().t() @ b[at:at + (1 << 18)].double()
    tol = (HALF_STEP[dtype] + (1 + 2.0 ** -8) * 5120 * 2.0 ** -23) * ref
    c = torch.tensor([n], dtype=torch.int32, device="cuda")
    dw = lm.grouped_gemm_dw(a, b, c, out_dtype=dtype)[0]
    worst = float(((dw.double() - ref).abs() / tol).max())
    assert worst <= 1.0, worst
    c = torch.tensor([16], dtype=torch.int32, device="cuda")
    at, bt = a.t().contiguous(), b.t().contiguous()
    for got in (lm.grouped_gemm(at, bt[None], c, out_dtype=dtype), lm.grouped_gemm_dx(at, b[None], c, out_dtype=dtype)):
        worst = float(((got.double() - ref).abs() / tol).max())
        assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_long_sums_of_one_sign_few_rows(dtype):
    """The same for the kernel of up to eight rows: 4096 products of a warp, then its sum in shared memory
    (2^22 / 4096 / warps of them), then the warps'; fewer than 1024 in all."""
    n = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(6)
    x = (torch.rand(5, n, generator=g, device="cuda") + 0.5).bfloat16()
    w = (torch.rand(24, n, generator=g, device="cuda") + 0.5).bfloat16()
    c = torch.tensor([5], dtype=torch.int32, device="cuda")
    ref = sum(x[:, at:at + (1 << 18)].double() @ w[:, at:at + (1 << 18)].double().t() for at in range(0, n, 1 << 18))
    tol = (HALF_STEP[dtype] + (1 + 2.0 ** -8) * 5120 * 2.0 ** -23) * ref
    worst = float(((lm.grouped_gemm(x, w[None], c, out_dtype=dtype).double() - ref).abs() / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("N", [24, 8200, 16008])  # eight warps, four with the ring, four without
@pytest.mark.parametrize("K", [4096, 32768 + 72])
def test_few_rows_past_a_drain(N, K):
    counts = [3, 0, 2]
    x, _, w, c = make(counts, N, K, rows=7)
    check_forward(lm.grouped_gemm(x, w, c, out_dtype=torch.float32), x, w, counts)


PENDING = """
import sys, torch
sys.path[:0] = [%r, %r]
import helpers as H
import synth
import latentmoe_layer_b200 as lm
from test_grouped_gpu import make
layer, _ = H.device_layer(synth.TINY)
x, dy, w, c = make([40, 0, 77], 136, 264)
few = make([3], 136, 264)
calls = [lambda: lm.grouped_gemm(x, w, c), lambda: lm.grouped_gemm_dw(dy, x, c), lambda: lm.quantize_fp8(x.repeat(1, 2)),
         lambda: lm.grouped_gemm(few[0], few[2], few[3])]
want = [f() for f in calls]
for f, y in zip(calls, want):
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    try:
        with torch.cuda.graph(graph, stream=stream, capture_error_mode="global"):
            s = lm.latentmoe_selftest_bounded_wait(layer.h)  # allocates, which a capture does not allow
    except Exception as e:
        pass
    assert s == lm.LMOE_ERR_CUDA, s
    got = f()
    torch.cuda.synchronize()
    for a, b in zip(got, y) if isinstance(y, tuple) else ((got, y),):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
print("not mine")
"""


def test_an_earlier_calls_error_is_not_reported():
    """An error that an earlier call of the library returned (here an allocation refused during a capture) is
    not this call's."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", PENDING % (here, os.path.dirname(here))], stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0 and "not mine" in r.stdout, r.stdout[-2000:]
