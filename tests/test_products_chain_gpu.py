"""The products one after another: launches that overlap their predecessor's end must still see all it wrote
and overwrite nothing it reads, in streams and in captured graphs; and operands beyond 2^31 elements."""
import pytest
import torch

import latentmoe_layer_b200 as lm
from test_fp8_gpu import check_product, recipe, same
from test_grouped_gpu import check_dw, check_dx, check_forward, make, spread

pytestmark = pytest.mark.gpu


class Chain:
    """A dozen calls per pass, each reading what the one before wrote; every buffer is used again by the next pass."""

    def __init__(self, rows, N, K, E, seed):
        counts = spread(rows, E, seed)
        self.x, _, self.w, self.c = make(counts, N, K, seed=seed)
        self.w.mul_(0.25 / K ** 0.5)
        self.x0 = self.x.clone()
        self.y = torch.empty(rows, N, device="cuda").bfloat16()
        self.dw = torch.zeros(E, N, K, device="cuda").bfloat16()

    def run(self, wait=lambda: None):
        out = []
        for _ in range(3):
            lm.grouped_gemm(self.x, self.w, self.c, out=self.y)
            wait()
            lm.grouped_gemm_dw(self.y, self.x, self.c, out=self.dw)
            wait()
            wq, ws = lm.quantize_fp8(self.dw, block_rows=128)
            wait()
            xq, xs = lm.quantize_fp8(self.x)
            wait()
            lm.gemm_fp8(xq, xs, wq, ws, counts=self.c, out=self.y)
            wait()
            out.append(lm.grouped_gemm_dx(self.y, self.w, self.c, out=self.x, out_dtype=torch.bfloat16).clone())
            wait()
            out.append(xq)
        return [self.y.clone(), self.dw.clone()] + [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in out]


@pytest.mark.parametrize("rows,N,K,E", [(5, 64, 128, 3), (8, 2064, 4112, 2), (4, 8200, 4112, 1), (131, 264, 208, 16), (1500, 520, 1040, 11)])
def test_chain_without_a_pause(rows, N, K, E):
    chain = Chain(rows, N, K, E, rows)
    want = chain.run(torch.cuda.synchronize)
    assert all(torch.isfinite(t.float()).all() for t in want) and want[1].any()
    for _ in range(20):
        chain.x.copy_(chain.x0)
        got = chain.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_chain_in_a_graph_with_a_second_stream():
    """Captured behind a join of two streams, followed by work of the second one."""
    a, b = Chain(5, 64, 128, 3, 1), Chain(700, 264, 528, 7, 2)
    want = a.run(torch.cuda.synchronize), b.run(torch.cuda.synchronize)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.x.copy_(b.x0)
            got_b = b.run()
        a.x.copy_(a.x0)
        got_a = a.run()
        torch.cuda.current_stream().wait_stream(side)
        both = lm.grouped_gemm(b.x, b.w, b.c)  # reads what the other stream wrote
        lm.grouped_gemm(a.x, a.w, a.c, out=a.y)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for w, g in zip(want, (got_a, got_b)):
        assert all(torch.equal(p, q) for p, q in zip(w, g))
    assert torch.equal(both, lm.grouped_gemm(b.x, b.w, b.c))


def test_weights_beyond_32_bits():
    """1024 experts of 1032 x 2056: the last experts lie 2^31 elements and more behind the first."""
    E, N, K = 1024, 1032, 2056
    for rows in ([3, 5], [700, 300]):  # few rows and many
        x, dy, w2, _ = make(rows, N, K)
        w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
        w[-2:] = w2
        c = torch.zeros(E, dtype=torch.int32, device="cuda")
        c[-2:] = torch.tensor(rows, dtype=torch.int32, device="cuda")
        check_forward(lm.grouped_gemm(x, w, c), x, w2, rows)
        check_dx(lm.grouped_gemm_dx(dy, w, c), dy, w2, rows)
        del w
        dw = lm.grouped_gemm_dw(dy, x, c)
        check_dw(dw[-2:], dy, x, rows)
        assert not dw[:-2].any()
        del dw


def test_row_pitch_beyond_32_bits():
    rows, N, K, pitch = 33000, 72, 64, 65552
    counts = [rows - 200, 0, 200]
    x, dy, w, c = make(counts, N, K)
    wide = torch.zeros(rows, pitch, dtype=torch.bfloat16, device="cuda")
    xs, out = wide[:, 8:8 + K], wide[:, 1024:1024 + N]
    xs.copy_(x)
    lm.grouped_gemm(xs, w, c, out=out)
    check_forward(out[-200:], x[-200:], w[2:], [200])
    check_dw(lm.grouped_gemm_dw(dy, xs, c)[2:], dy[-200:], x[-200:], [200])
    assert not wide[:, :8].any() and not wide[:, 8 + K:1024].any() and not wide[:, 1024 + N:2048].any()


def test_8_bit_operands_beyond_32_bits():
    rows, N, K = 66000, 72, 32784
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, K, generator=g, device="cuda", dtype=torch.bfloat16)
    xq, xs = lm.quantize_fp8(x)
    same((xq[-40:], xs[-40:]), recipe(x[-40:], 1))
    same((xq[:40], xs[:40]), recipe(x[:40], 1))
    wq, ws = lm.quantize_fp8(x[:N], block_rows=128)
    y = lm.gemm_fp8(xq, xs, wq, ws)
    check_product(y[-300:], xq[-300:], xs[-300:], wq, ws, [300])
    many, blocks = lm.quantize_fp8(x, block_rows=128)
    same((many[-80:], blocks[-1:]), recipe(x[-80:], 128))  # 66000 = 515 * 128 + 80
