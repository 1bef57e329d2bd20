"""The products beside autograd."""
import pytest
import torch

import latentmoe_layer_b200 as lm
from test_grouped_gpu import make

pytestmark = pytest.mark.gpu
COUNTS, N, K = [37, 0, 90, 2], 136, 200


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
