"""Device waits of the products that run out. A limit of a few polls makes valid calls give up at places that
differ from run to run, with loads and MMAs in flight. The kernel has to end, the report to reach every thread
once, and calls after it to be right. Each case runs in a child process: the limit is process-wide."""
import os
import subprocess
import sys
import threading

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
DEFAULT = 1 << 24

# counts, N, K of each form of the kernel; tiles, k-blocks (and partial ones) enough for all stages
FORMS = {
    "forward": ([300, 0, 77, 513], 520, 1032),
    "forward, two pairs share": ([40, 200], 2568, 2056),
    "forward, four pairs share": ([40], 264, 4096),
    "dx": ([300, 0, 77, 513], 1032, 520),
    "dx, four pairs share": ([30, 9], 2952, 264),
    "dw": ([300, 0, 77, 513, 1000], 520, 264),
    "fp8": ([20, 0, 33, 41], 520, 1040),
    "fp8, four pairs share": ([40], 264, 4096),
    "fp8, rows on M": ([300, 0, 77, 513], 520, 1040),
}


def launcher(form):
    import torch
    import latentmoe_layer_b200 as lm
    from test_fp8_gpu import operands
    from test_grouped_gpu import make
    counts, N, K = FORMS[form]
    if form.startswith("fp8"):
        xq, xs, wq, ws, c = operands(counts, N, K)
        return lambda: lm.gemm_fp8(xq, xs, wq, ws, counts=c, out_dtype=torch.float32)
    x, dy, w, c = make(counts, N, K)
    if form.startswith("forward"):
        return lambda: lm.grouped_gemm(x, w, c, out_dtype=torch.float32)
    if form.startswith("dx"):
        return lambda: lm.grouped_gemm_dx(dy, w, c, out_dtype=torch.float32)
    return lambda: lm.grouped_gemm_dw(dy, x, c, out_dtype=torch.float32)


def child_form(form):
    import torch
    import latentmoe_layer_b200 as lm
    run = launcher(form)
    want = run()
    assert lm.latentmoe_products_status() == lm.LMOE_OK
    gave_up = 0
    for limit in (0, 0, 1, 2, 5, 0, 20, 100, 0):
        for _ in range(4):
            lm.latentmoe_set_products_wait_limit(limit)
            got = run()
            torch.cuda.synchronize()
            lm.latentmoe_set_products_wait_limit(DEFAULT)
            s = lm.latentmoe_products_status()
            assert s in (lm.LMOE_OK, lm.LMOE_ERR_TIMEOUT)
            assert s == lm.LMOE_ERR_TIMEOUT or limit > 0  # the first wait for operands cannot have been over
            assert s == lm.LMOE_ERR_TIMEOUT or torch.equal(got, want)
            gave_up += s == lm.LMOE_ERR_TIMEOUT
            again = run()
            torch.cuda.synchronize()
            assert torch.equal(again, want) and lm.latentmoe_products_status() == lm.LMOE_OK
    print("gave up in %d of 36" % gave_up)


def child_reports():
    """One timeout: every thread is told once, by a call that does no work or by the status."""
    import torch
    import latentmoe_layer_b200 as lm
    from test_grouped_gpu import make
    x, _, w, c = make([300, 77], 264, 520)
    want = lm.grouped_gemm(x, w, c)
    told, start, go = [], threading.Event(), threading.Event()

    def other():
        lm.grouped_gemm(x, w, c)
        start.set()
        go.wait(60)
        try:
            lm.grouped_gemm(x, w, c)
        except lm.LmoeError as e:
            told.append(e.status)
        told.append(torch.equal(lm.grouped_gemm(x, w, c), want))

    t = threading.Thread(target=other)
    t.start()
    assert start.wait(60)
    lm.latentmoe_set_products_wait_limit(0)
    lm.grouped_gemm(x, w, c)
    lm.latentmoe_set_products_wait_limit(DEFAULT)
    torch.cuda.synchronize()
    out = torch.full_like(want, -7.0)
    try:
        lm.grouped_gemm(x, w, c, out=out)
        raise AssertionError("the timeout was not reported")
    except lm.LmoeError as e:
        assert e.status == lm.LMOE_ERR_TIMEOUT
    torch.cuda.synchronize()
    assert (out == -7).all()  # the call that reports launches nothing
    assert torch.equal(lm.grouped_gemm(x, w, c), want)
    go.set()
    t.join()
    assert told == [lm.LMOE_ERR_TIMEOUT, True], told
    assert lm.latentmoe_products_status() == lm.LMOE_OK


def child_streams():
    """Calls that are in flight beside one that gives up, and graphs replayed after it, are right."""
    import torch
    import latentmoe_layer_b200 as lm
    from test_grouped_gpu import make
    x, _, w, c = make([3000, 2077, 4000], 1032, 2056)
    want = lm.grouped_gemm(x, w, c)
    out, bad_out = torch.empty_like(want), torch.empty_like(want)
    graph, bad_graph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.grouped_gemm(x, w, c, out=out)
    lm.latentmoe_set_products_wait_limit(0)
    with torch.cuda.graph(bad_graph):
        lm.grouped_gemm(x, w, c, out=bad_out)
    lm.latentmoe_set_products_wait_limit(DEFAULT)
    side = torch.cuda.Stream()
    for _ in range(10):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            bad_graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert lm.latentmoe_products_status() == lm.LMOE_ERR_TIMEOUT
        assert torch.equal(out, want)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and lm.latentmoe_products_status() == lm.LMOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["reports", "streams"] + list(FORMS))
def test_waits_that_run_out(case):
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True, timeout=300)
    assert r.returncode == 0 and "case ok" in r.stdout, r.stdout[-3000:]


if __name__ == "__main__":
    sys.path[:0] = [HERE, os.path.dirname(HERE)]
    if sys.argv[1] in FORMS:
        child_form(sys.argv[1])
    else:
        globals()["child_" + sys.argv[1]]()
    print("case ok")
