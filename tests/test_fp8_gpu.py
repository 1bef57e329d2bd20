"""The 8-bit quantiser (bit for bit against its recipe) and the block-scaled product (against fp64).

Tolerance of the product, derived: block sums of 128 exact products accumulated in fp32 (128 * 2^-23
of sum |a b|), the scales' product rounded once (2^-24), one fused multiply-add per block: together
at most (128 + 2 + blocks) * 2^-23 * sum |s a b|; rounding the result adds half a step of its value.
"""
import numpy as np
import pytest
import torch

import latentmoe_layer_b200 as lm
from test_grouped_gpu import HALF_STEP, LARGE_GRIDS, spread

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def recipe(x, block):
    """(code bytes, scales) by the recipe, on the CPU in IEEE fp32."""
    x = x.float().cpu()
    *lead, R, K = x.shape
    rb, kb = -(-R // block), -(-K // 128)
    pad = torch.zeros(*lead, rb * block, kb * 128)
    pad[..., :R, :K] = x
    pad = pad.reshape(*lead, rb, block, kb, 128)
    a = pad.abs().amax(dim=(-3, -1)).clamp(min=2.0 ** -100)
    q = pad * (torch.tensor(448.0) / a)[..., :, None, :, None]
    q = torch.where(q.isfinite(), q.clamp(-448, 448), q)  # saturating
    codes = q.reshape(*lead, rb * block, kb * 128)[..., :R, :K].contiguous().to(F8)
    return codes.view(torch.uint8), a / 448.0


def same(got, want):
    codes, scales = got
    wc, wsc = want
    gc, gs = codes.cpu().view(torch.uint8), scales.cpu()
    nan = (wc & 0x7F) == 0x7F  # a NaN's sign is not specified
    assert torch.equal(gc & 0x7F == 0x7F, nan) and torch.equal(gc[~nan], wc[~nan])
    assert torch.equal(gs.isnan(), wsc.isnan()) and torch.equal(gs[~gs.isnan()], wsc[~wsc.isnan()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,K", [(1, 16), (1, 128), (3, 144), (64, 256), (129, 400), (257, 1040), (1000, 2048)])
def test_quantize_rows(R, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(R * 1000 + K)
    x = (torch.randn(R, K, generator=g, device="cuda") * torch.randn(R, 1, generator=g, device="cuda").exp()).to(dtype)
    codes, scales = lm.quantize_fp8(x)
    assert codes.dtype == F8 and codes.shape == x.shape and scales.shape == (R, -(-K // 128))
    same((codes, scales), recipe(x, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (130, 144), (3, 300, 400), (2, 127, 1040)])
def test_quantize_blocks(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = (torch.randn(*shape, generator=g, device="cuda") * 0.02).to(dtype)
    codes, scales = lm.quantize_fp8(x, block_rows=128)
    assert scales.shape == (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128))
    same((codes, scales), recipe(x, 128))


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_special_values(block):
    """Zero blocks, tiny, huge and non-finite values: each stays in its block."""
    x = torch.randn(256, 512, device="cuda")
    x[0, :128] = 0
    x[1, :128] = 1e-35
    x[2, 128:256] = 3e38
    x[3, 5] = float("nan")
    x[130, 300] = float("inf")
    x[131, 400] = -float("inf")
    x[132, 0:128] *= 2.0 ** -120
    x[133, :] = 1e-45
    x[140, 7] = -0.0
    same(lm.quantize_fp8(x, block_rows=block), recipe(x, block))
    same(lm.quantize_fp8(x.bfloat16(), block_rows=block), recipe(x.bfloat16(), block))


def test_quantize_ties_and_saturation():
    """Values on the e4m3 grid come back as they are, midpoints go to the even code."""
    grid = torch.arange(0, 127, dtype=torch.uint8).view(F8).float()  # 0 .. 448
    mids = (grid[1:] + grid[:-1]) / 2
    x = torch.zeros(4, 128)
    x[0, :127], x[1, :126], x[2, :127], x[3, :126] = grid, mids, -grid, -mids
    x[1, 127] = x[3, 127] = 448.0
    codes, scales = lm.quantize_fp8(x.cuda())
    assert torch.equal(scales.cpu(), torch.ones(4, 1))
    same((codes, scales), recipe(x, 1))
    assert torch.equal(codes[0, :127].float().cpu(), grid)


def test_quantize_row_pitch_and_empty():
    wide = torch.randn(33, 400, device="cuda").bfloat16()
    x = wide[:, 16:16 + 256]
    same(lm.quantize_fp8(x), recipe(x, 1))
    same(lm.quantize_fp8(x, block_rows=128), recipe(x, 128))
    codes, scales = lm.quantize_fp8(wide[:0])
    assert codes.shape == (0, 400) and scales.shape == (0, 4)


def operands(counts, N, K, rows=None, seed=0, dense=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = sum(counts) if rows is None else rows
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.randn(rows, 1, generator=g, device="cuda").exp()
    w = torch.randn(len(counts), N, K, generator=g, device="cuda") * 0.02
    xq, xs = lm.quantize_fp8(x)
    wq, ws = lm.quantize_fp8(w, block_rows=128)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    return (xq, xs, wq[0], ws[0], None) if dense else (xq, xs, wq, ws, c)


def check_product(y, xq, xs, wq, ws, counts):
    if wq.dim() == 2:
        wq, ws = wq[None], ws[None]
    _, N, K = wq.shape
    col = torch.arange(K, device="cuda") // 128
    row = torch.arange(N, device="cuda") // 128
    at = 0
    for e, n in enumerate(counts):
        if n:
            a = xq[at:at + n].double() * xs[at:at + n].double()[:, col]
            b = wq[e].double() * ws[e].double()[row][:, col]
            ref, mag = a @ b.t(), a.abs() @ b.abs().t()
            got = y[at:at + n]
            assert torch.isfinite(got).all()
            tol = HALF_STEP[y.dtype] * ref.abs() + (1 + 2.0 ** -8) * (130 + ws.shape[-1]) * 2.0 ** -23 * mag + 1e-38
            worst = float(((got.double() - ref).abs() / tol).max())
            assert worst <= 1.0, worst
        at += n


CASES = [
    ([1] + [0] * 500 + [3, 0, 1], 40, 1040), ([0, 8], 136, 2048), ([9], 136, 2048), ([1] * 8, 72, 528), ([4, 0, 5], 264, 80),
    ([5], 8, 16), ([1], 128, 128), ([0, 0, 3, 0], 136, 64), ([31, 32, 33, 0, 1], 264, 144), ([64, 63, 65, 128], 520, 656),
    ([255, 256, 257], 256, 512), ([513, 0, 130, 700], 384, 1040), ([300], 2048, 2560), (spread(1031, 37, 1), 264, 464),
    (spread(40, 128, 2), 512, 512), (spread(333, 1024, 3, empty=0.7), 40, 48),
    ([40], 264, 4096), ([20, 0, 30], 136, 4112), ([100], 520, 4096), ([60, 61, 0, 62], 520, 4368),  # shared contractions
]


@pytest.mark.parametrize("counts,N,K", CASES, ids=["%dx%d e%d r%d" % (n, k, len(c), sum(c)) for c, n, k in CASES])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_grouped_product(counts, N, K, dtype):
    xq, xs, wq, ws, c = operands(counts, N, K)
    y = lm.gemm_fp8(xq, xs, wq, ws, counts=c, out_dtype=dtype)
    assert y.dtype == dtype and y.shape == (sum(counts), N)
    check_product(y, xq, xs, wq, ws, counts)


@pytest.mark.parametrize("rows,N,K", [(1, 8, 16), (1, 1024, 2048), (2, 136, 400), (17, 640, 8192), (33, 2560, 1040),
                                      (64, 264, 4096), (129, 5120, 256), (700, 1288, 2064), (2049, 512, 1024)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_dense_product(rows, N, K, dtype):
    xq, xs, wq, ws, _ = operands([rows], N, K, dense=True)
    y = lm.gemm_fp8(xq, xs, wq, ws, out_dtype=dtype)
    check_product(y, xq, xs, wq, ws, [rows])


@pytest.mark.parametrize("zero_tail", [False, True])
def test_rows_behind_the_last_group(zero_tail):
    for counts, rows, N, K in (([40, 0, 300, 17], 700, 136, 272), ([20, 0, 9], 60, 264, 4112), ([100, 900], 1400, 264, 272)):
        used = sum(counts)
        xq, xs, wq, ws, c = operands(counts, N, K, rows=rows)
        xq.view(torch.uint8)[used:] = 0x7F  # NaN codes and scales in rows that nobody may read into a result
        xs[used:] = float("nan")
        y = torch.full((rows, N), -7.0, device="cuda").bfloat16()
        lm.gemm_fp8(xq, xs, wq, ws, counts=c, out=y, zero_tail=zero_tail)
        check_product(y, xq, xs, wq, ws, counts)
        assert (y[used:] == (0.0 if zero_tail else -7.0)).all()


@pytest.mark.parametrize("counts,rows", [([0, 1, 0], 8), ([0, 0], 5), ([2, 0, 3], 8)])
def test_few_rows_and_a_tail(counts, rows):
    N, K = 264, 528
    xq, xs, wq, ws, c = operands(counts, N, K, rows=rows)
    used = sum(counts)
    xq.view(torch.uint8)[used:] = 0x7F
    xs[used:] = float("nan")
    for zero_tail in (False, True):
        y = torch.full((rows, N), -7.0, device="cuda")
        lm.gemm_fp8(xq, xs, wq, ws, counts=c, out=y, zero_tail=zero_tail)
        check_product(y, xq, xs, wq, ws, counts)
        assert (y[used:] == (0.0 if zero_tail else -7.0)).all()


@pytest.mark.parametrize("counts,N,K", LARGE_GRIDS, ids=["%dx%d e%d r%d" % (n, k, len(c), sum(c)) for c, n, k in LARGE_GRIDS])
def test_few_rows_on_large_grids(counts, N, K):
    K += K % 16
    used = sum(counts)
    rows = min(8, used + 1)
    xq, xs, wq, ws, c = operands(counts, N, K, rows=rows)
    xq.view(torch.uint8)[used:] = 0x7F
    xs[used:] = float("nan")
    for zero_tail in (False, True):
        y = torch.full((rows, N), -7.0, device="cuda")
        lm.gemm_fp8(xq, xs, wq, ws, counts=c, out=y, zero_tail=zero_tail)
        check_product(y, xq, xs, wq, ws, counts)
        assert (y[used:] == (0.0 if zero_tail else -7.0)).all()
    if len(counts) == 1:
        check_product(lm.gemm_fp8(xq[:used], xs[:used], wq[0], ws[0]), xq[:used], xs[:used], wq[0], ws[0], counts)


def test_bad_values_stay_in_their_rows():
    counts, N, K = [70, 33, 100], 136, 272
    xq, xs, wq, ws, c = operands(counts, N, K)
    xq.view(torch.uint8)[70:103, 200] = 0x7F
    y = lm.gemm_fp8(xq, xs, wq, ws, counts=c)
    assert y[70:103].isnan().all()
    check_product(y[:70], xq[:70], xs[:70], wq, ws, [70, 0, 0])
    check_product(y[103:], xq[103:], xs[103:], wq, ws, [0, 0, 100])


def test_output_pitch_and_no_rows():
    xq, xs, wq, ws, c = operands([9, 30], 136, 272)
    wide = torch.full((39, 136 + 24), 5.0, device="cuda").bfloat16()
    y = lm.gemm_fp8(xq, xs, wq, ws, counts=c, out=wide[:, 8:144])
    check_product(y, xq, xs, wq, ws, [9, 30])
    assert (wide[:, :8] == 5).all() and (wide[:, 144:] == 5).all()
    assert lm.gemm_fp8(xq[:0], xs[:0], wq, ws, counts=c).shape == (0, 136)


def test_same_bits_on_two_streams_and_in_a_graph():
    xq, xs, wq, ws, c = operands(spread(1500, 11, 5), 520, 1040)
    first = lm.gemm_fp8(xq, xs, wq, ws, counts=c)
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            got.append(lm.gemm_fp8(xq, xs, wq, ws, counts=c))
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.gemm_fp8(xq, xs, wq, ws, counts=c, out=out)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for g in got + [out]:
        assert torch.equal(first, g)


def test_serving_an_expert_layer_in_8_bits():
    """Quantised rows through up, relu2, requantised, down: close to the bf16 products of the same weights."""
    counts, L, I = [6, 0, 1, 25], 256, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(32, L, generator=g, device="cuda").bfloat16()
    up = (torch.randn(4, I, L, generator=g, device="cuda") * 0.1).bfloat16()
    down = (torch.randn(4, L, I, generator=g, device="cuda") * 0.1).bfloat16()
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    uq, dq = lm.quantize_fp8(up, block_rows=128), lm.quantize_fp8(down, block_rows=128)
    h = lm.gemm_fp8(*lm.quantize_fp8(x), *uq, counts=c)
    y = lm.gemm_fp8(*lm.quantize_fp8(torch.relu(h).square()), *dq, counts=c)
    hb = lm.grouped_gemm(x, up, c)
    yb = lm.grouped_gemm(torch.relu(hb).square(), down, c)
    # x, up, a and down are each rounded to e4m3 (2^-4 at most, of the value): the square doubles the
    # first two, so at most 6 * 2^-4 of the terms' norm, the errors being independent of their signs
    assert float((y.float() - yb.float()).norm() / yb.float().norm()) < 6 * 2.0 ** -4


def test_refusals_of_the_binding():
    xq, xs, wq, ws, c = operands([3, 5], 136, 272)
    bad = [lambda: lm.quantize_fp8(torch.zeros(4, 32, device="cuda").half()), lambda: lm.quantize_fp8(torch.zeros(32, device="cuda")),
           lambda: lm.quantize_fp8(torch.zeros(4, 32, device="cuda"), block_rows=64),
           lambda: lm.quantize_fp8(torch.zeros(32, 16, device="cuda").t()),
           lambda: lm.quantize_fp8(torch.zeros(2, 8, 64, device="cuda")[:, :, :32]),
           lambda: lm.gemm_fp8(xq, xs, wq, ws), lambda: lm.gemm_fp8(xq, xs, wq[0], ws[0], counts=c),
           lambda: lm.gemm_fp8(xq, xs[:, :2], wq, ws, counts=c), lambda: lm.gemm_fp8(xq, xs, wq, ws[:, :1], counts=c),
           lambda: lm.gemm_fp8(xq.view(torch.uint8), xs, wq, ws, counts=c), lambda: lm.gemm_fp8(xq, xs.double(), wq, ws, counts=c),
           lambda: lm.gemm_fp8(xq, xs, wq, ws, counts=c[:1]), lambda: lm.gemm_fp8(xq, xs.cpu(), wq, ws, counts=c),
           lambda: lm.gemm_fp8(xq[:, :256], xs, wq, ws, counts=c), lambda: lm.gemm_fp8(xq, xs, wq, ws, counts=c, out_dtype=torch.half)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lm.LmoeError) as e:
        lm.quantize_fp8(torch.zeros(4, 24, device="cuda"))
    assert e.value.status == lm.LMOE_ERR_UNSUPPORTED
