"""Measured cases of the expert products: grouped by expert with ragged sizes (forward and gradients),
and in 8-bit floating point with one scale per block of 128.

``run`` computes a case in its plain form (elementary torch operations in fp32), or, where ``own`` is
true, with the library's operators. Four operators:

  grouped   y[r] = x[r] W[e(r)]^T, rows in expert order, per-expert row counts on the device
  gradient  dx[r] = dy[r] W[e(r)] and dW[e] = sum of dy[r]^T x[r] over the expert's rows
  quantize  e4m3 codes and fp32 scales: one scale per 1 x 128 block of a row (activations) or per
            128 x 128 block of a matrix (weights); a = max(amax, 2^-100), scale = a / 448,
            code = e4m3(x * (448 / a)), every step an fp32 operation rounded to nearest
  fp8       y[r, n] = sum over blocks b of sx[r, b] sw[e, n / 128, b] * (codes' product over block b)
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
TINY = 2.0 ** -100


def listed():
    return [
        # the smallest layer's up projection: 64 tokens, two experts each; the call's latency is what counts
        {"name": "grouped, smallest layer", "op": "grouped", "E": 16, "rows": 128, "N": 128, "K": 64, "f32": False},
        # a decode step of 128 tokens, 8 of 128 experts each: every expert's weights are read for a handful of rows
        {"name": "grouped, decode", "op": "grouped", "E": 128, "rows": 1024, "N": 2560, "K": 2048, "f32": False},
        # a prompt of 2048 tokens, 22 experts each over 64 experts: uneven groups of about 700 rows
        {"name": "grouped, prompt", "op": "grouped", "E": 64, "rows": 45056, "N": 5120, "K": 2048, "f32": False},
        # gradients of a small layer with an odd number of rows
        {"name": "gradient, small and odd", "op": "gradient", "E": 16, "rows": 131, "N": 264, "K": 200, "f32": True},
        # gradients of a short training batch: the weights and their gradient are most of the traffic
        {"name": "gradient, short batch", "op": "gradient", "E": 128, "rows": 8192, "N": 2560, "K": 2048, "f32": False},
        # gradients of the down projection for a full training batch, weight gradient in fp32
        {"name": "gradient, training batch", "op": "gradient", "E": 64, "rows": 45056, "N": 2048, "K": 5120, "f32": True},
        # a decode step's hidden states before an 8-bit product
        {"name": "quantize, decode rows", "op": "quantize", "mats": 1, "rows": 64, "K": 8192, "block": 1, "f32": False},
        # a prompt's hidden states before an 8-bit product
        {"name": "quantize, prompt rows", "op": "quantize", "mats": 1, "rows": 16384, "K": 8192, "block": 1, "f32": False},
        # one token through a dense projection (the shared expert's up projection)
        {"name": "fp8, one token", "op": "fp8", "E": 0, "rows": 1, "N": 10240, "K": 8192, "f32": False},
        # a decode step over 128 experts with 8-bit weights
        {"name": "fp8, grouped decode", "op": "fp8", "E": 128, "rows": 1024, "N": 2560, "K": 2048, "f32": False},
        # a prompt through uneven groups
        {"name": "fp8, grouped prompt", "op": "fp8", "E": 64, "rows": 45056, "N": 5120, "K": 2048, "f32": False},
        # a prompt through the shared expert's up projection
        {"name": "fp8, dense prompt", "op": "fp8", "E": 0, "rows": 16384, "N": 10240, "K": 8192, "f32": False},
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in lo .. hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    top = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["grouped", "gradient", "quantize", "fp8"])
        f32 = rng.random() < 0.3
        if op == "quantize":
            block = rng.choice([1, 1, 128])
            case = {"op": op, "mats": 1 if block == 1 else _log(rng, 1, 64, 1), "rows": _log(rng, 1, 16384, 1),
                    "K": _log(rng, 64, 10240, 16), "block": block, "f32": f32}
        else:
            dense = op == "fp8" and rng.random() < 0.4
            step = 16 if op == "fp8" else 8
            case = {"op": op, "E": 0 if dense else _log(rng, 1, 256, 1), "rows": _log(rng, 1, 45056, 1),
                    "N": _log(rng, 64, 10240, 8), "K": _log(rng, 64, 10240, step), "f32": f32}
            e = max(1, case["E"])
            if e * case["N"] * case["K"] > 128 * 2560 * 2048:
                continue  # beyond the largest layer's weights listed
            if e > 1 and (case["rows"] + 64 * e) * (case["N"] + case["K"]) > 6 * 45056 * 7168:
                continue  # the padded plain form would not fit beside its inputs
        w = work(case)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return case


def _counts(case, seed):
    """Rows per expert as a router leaves them: uneven, about a tenth of the experts without any."""
    E, rows = case["E"], case["rows"]
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    p = torch.exp(0.5 * torch.randn(E, generator=g))
    p = torch.where(torch.rand(E, generator=g) < 0.1, torch.zeros(E), p)
    if float(p.sum()) == 0.0:
        p = torch.ones(E)
    picks = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(picks, minlength=E).to(torch.int32)


def _quantize_plain(x, block):
    """(codes, scales) of x [..., R, K] with one scale per block x 128 elements."""
    *lead, R, K = x.shape
    rb, kb = -(-R // block), -(-K // 128)
    v = x.float()
    pad = torch.nn.functional.pad(v, (0, kb * 128 - K, 0, rb * block - R))
    pad = pad.reshape(*lead, rb, block, kb, 128)
    a = pad.abs().amax(dim=(-3, -1)).clamp(min=TINY)
    inv = 448.0 / a
    codes = (pad * inv[..., :, None, :, None]).reshape(*lead, rb * block, kb * 128)[..., :R, :K].contiguous().to(FP8)
    return codes, a / 448.0


def _dequantize_plain(codes, scales, block):
    *lead, R, K = codes.shape
    s = scales.repeat_interleave(128, dim=-1)[..., :K]
    if block > 1:
        s = s.repeat_interleave(block, dim=-2)[..., :R, :]
    return codes.float() * s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    out = torch.float32 if case["f32"] else torch.bfloat16
    st = {"case": case, "out": out}
    if case["op"] == "quantize":
        shape = (case["rows"], case["K"]) if case["block"] == 1 else (case["mats"], case["rows"], case["K"])
        st["x"] = normal(*shape, dtype=out)
        # rows of different size, as hidden states have
        st["x"].mul_(torch.exp(normal(*shape[:-1], 1, dtype=torch.float32)).to(out))
        return st
    E, R, N, K = case["E"], case["rows"], case["N"], case["K"]
    if E:
        counts = _counts(case, seed)
        st["cap"] = int(counts.max())   # what the plain form pads each expert to
        st["counts"] = counts.to(dev)
    x = normal(R, K)
    w = normal(*((E, N, K) if E else (N, K)), scale=0.02)
    if case["op"] == "fp8":
        st["xq"], st["xs"] = _quantize_plain(x, 1)
        # the weights' codes and scales, matrix by matrix as a checkpoint is converted
        parts = [_quantize_plain(m, 128) for m in (w if E else w[None])]
        st["wq"] = torch.stack([p[0].view(torch.uint8) for p in parts]).view(FP8)
        st["ws"] = torch.stack([p[1] for p in parts])
        if not E:
            st["wq"], st["ws"] = st["wq"][0], st["ws"][0]
        return st
    st["w"], st["x"] = w, x
    if case["op"] == "gradient":
        st["dy"] = normal(R, N)
    return st


def _slots(counts, rows, cap):
    """Expert and position of every row, and the row and validity of every padded place."""
    ends = counts.long().cumsum(0)
    starts = ends - counts
    r = torch.arange(rows, device=counts.device)
    e = torch.searchsorted(ends, r, right=True)
    at = torch.arange(cap, device=counts.device)
    place = (starts[:, None] + at).clamp(max=rows - 1)
    return e, r - starts[e], place, at < counts[:, None]


def _padded(v, place, valid):
    return torch.where(valid[..., None], v.float()[place], 0.0)


def _run_plain(st):
    c, out = st["case"], st["out"]
    if c["op"] == "quantize":
        return list(_quantize_plain(st["x"], c["block"]))
    if c["op"] == "fp8":
        x = _dequantize_plain(st["xq"], st["xs"], 1)
        w = _dequantize_plain(st["wq"], st["ws"], 128)
        if not c["E"]:
            return (x @ w.t()).to(out)
    else:
        x, w = st["x"], st["w"].float()
    e, pos, place, valid = _slots(st["counts"], c["rows"], st["cap"])
    xp = _padded(x, place, valid)
    if c["op"] != "gradient":
        return torch.bmm(xp, w.transpose(1, 2))[e, pos].to(out)
    dyp = _padded(st["dy"], place, valid)
    return {"dx": torch.bmm(dyp, w)[e, pos].to(torch.bfloat16), "dw": torch.bmm(dyp.transpose(1, 2), xp).to(out)}


def _run_own(st):
    import latentmoe_layer_b200 as lm
    c, out = st["case"], st["out"]
    if c["op"] == "quantize":
        return list(lm.quantize_fp8(st["x"], block_rows=c["block"]))
    if c["op"] == "fp8":
        return lm.gemm_fp8(st["xq"], st["xs"], st["wq"], st["ws"], counts=st.get("counts"), out_dtype=out)
    if c["op"] == "grouped":
        return lm.grouped_gemm(st["x"], st["w"], st["counts"], out_dtype=out)
    return {"dx": lm.grouped_gemm_dx(st["dy"], st["w"], st["counts"]),
            "dw": lm.grouped_gemm_dw(st["dy"], st["x"], st["counts"], out_dtype=out)}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    f = 4 if case["f32"] else 2
    K, R = case["K"], case["rows"]
    if case["op"] == "quantize":
        n = case["mats"] * R * K
        scales = case["mats"] * -(-R // case["block"]) * -(-K // 128)
        return {"bytes": n * (f + 1) + 4 * scales, "flops": 3 * n}
    N, E = case["N"], max(1, case["E"])
    # experts that have rows: those of a tenth have none by construction, and few rows hit few experts
    hit = E if not case["E"] else max(1.0, 0.9 * E * (1.0 - math.exp(-R / (0.9 * E))))
    if case["op"] == "grouped":
        return {"bytes": 2 * R * K + 2 * hit * N * K + f * R * N + 4 * E, "flops": 2 * R * N * K}
    if case["op"] == "gradient":
        return {"bytes": 2 * R * (N + K) + 2 * hit * N * K + 2 * R * K + f * E * N * K + 4 * E, "flops": 4 * R * N * K}
    kb = -(-K // 128)
    return {"bytes": R * K + 4 * R * kb + hit * (N * K + 4 * kb * -(-N // 128)) + f * R * N + 4 * E, "flops": 2 * R * N * K}


def exact(case, seed):
    """The definition in fp64, expert by expert."""
    st = prepare(case, seed)
    if case["op"] == "quantize":
        x = st["x"].double()
        step = case["block"]
        chunk = step if step > 1 else 4096
        codes, scales = [], []
        for r in range(0, x.shape[-2], chunk):
            rows = x[..., r:r + chunk, :]
            cc, ss = [], []
            for k in range(0, x.shape[-1], 128):
                b = rows[..., k:k + 128]
                a = b.abs().amax(-1, keepdim=True)
                if step > 1:
                    a = a.amax(-2, keepdim=True)
                a = a.clamp(min=TINY)
                cc.append((b / (a / 448.0)).float().to(FP8).view(torch.uint8))
                ss.append(a.squeeze(-1) / 448.0)
            codes.append(torch.cat(cc, -1))
            scales.append(torch.stack(ss, -1))
        return [torch.cat(codes, -2).view(FP8), torch.cat(scales, -2)]
    R, N, K = case["rows"], case["N"], case["K"]
    ends = st["counts"].tolist() if case["E"] else [R]
    if case["op"] == "fp8":
        wq, ws = (st["wq"], st["ws"]) if case["E"] else (st["wq"][None], st["ws"][None])

        def expert(e):
            col = torch.arange(K, device="cuda") // 128
            row = torch.arange(N, device="cuda") // 128
            return wq[e].double() * ws[e].double()[row][:, col]

        col = torch.arange(K, device="cuda") // 128
        y = torch.zeros(R, N, dtype=torch.float64, device="cuda")
        at = 0
        for e, n in enumerate(ends):
            if n:
                xe = st["xq"][at:at + n].double() * st["xs"][at:at + n].double()[:, col]
                y[at:at + n] = xe @ expert(e).t()
            at += n
        return y
    y = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    dx = torch.zeros(R, K, dtype=torch.float64, device="cuda")
    dw = torch.zeros(case["E"], N, K, dtype=torch.float64, device="cuda") if case["op"] == "gradient" else None
    at = 0
    for e, n in enumerate(ends):
        if n:
            we = st["w"][e].double()
            xe = st["x"][at:at + n].double()
            if case["op"] == "grouped":
                y[at:at + n] = xe @ we.t()
            else:
                de = st["dy"][at:at + n].double()
                dx[at:at + n] = de @ we
                dw[e] = de.t() @ xe
        at += n
    return y if case["op"] == "grouped" else {"dx": dx, "dw": dw}
