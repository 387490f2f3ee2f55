"""Cases that measure the operators of an 8-bit linear layer: the root-mean-square
norm with the residual's addition (its output in 16 or 32 bits, or in 8 bits with
scales) and its gradient, the quantisation in blocks of 128, and the matrix
product of 8-bit operands with a scale for each block of 128 along K.

``listed()`` and ``draw()`` give cases (dicts of plain values), ``prepare()``
the tensors a training or serving program has in hand, ``run()`` one pass.
Where the module's ``own`` is false ``run`` computes with elementary torch
operations in fp32; where it is true it calls recsys_linear_layers_amd.

Case keys: ``op`` (norm, norm8, norm_grad, quant, gemm8), ``type`` (of the 16- or
32-bit tensors, C among them), ``q`` (the 8-bit type; of A for gemm8), and the
sizes: ``N`` rows, ``D`` columns, ``pad``: extra elements between rows; ``M``,
``N``, ``K`` of C = A B^T; ``squares``: 128 x 128 blocks (of B for gemm8), else
128 consecutive values of a row; ``residual``: whether a residual is added;
``forms``: which forms quant gives (plain, transposed, both).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
BLOCK = 128
SMALLEST_SCALE = 2.0 ** -126


def listed():
    return [
        # one decode step of one sequence: the latency of a single row in front of an 8-bit product
        dict(name="norm8-one-row", op="norm8", type="bf16", q="e4m3", N=1, D=8192, pad=0, residual=True),
        # the same in front of the 16384 x 28672 x 8192 feed-forward product
        dict(name="norm8-batch", op="norm8", type="bf16", q="e4m3", N=16384, D=8192, pad=0, residual=True),
        # a layer whose products stay in 16 bits, odd sizes, rows at an odd distance
        dict(name="norm-odd", op="norm", type="f16", N=8191, D=5003, pad=3, residual=True),
        # the gradient of the batch, joined with the residual's own
        dict(name="norm-grad-batch", op="norm_grad", type="bf16", N=16384, D=8192, pad=0, residual=True),
        # the gradient in full precision, odd sizes
        dict(name="norm-grad-odd", op="norm_grad", type="f32", N=8191, D=5003, pad=3, residual=False),
        # a weight after its update: for the forward product, and transposed for the inputs' gradient
        dict(name="quant-weight", op="quant", type="bf16", q="e4m3", N=28672, D=8192, pad=0, squares=True, forms="both"),
        # odd activations on their way into a product and into the weight's gradient
        dict(name="quant-odd", op="quant", type="f16", q="e4m3", N=8191, D=5003, pad=3, squares=False, forms="both"),
        # one decode step: the weight's bytes
        dict(name="gemm8-one-token", op="gemm8", type="bf16", q="e4m3", M=1, N=28672, K=8192, squares=True),
        # a small batch of sequences, odd sizes
        dict(name="gemm8-few-odd", op="gemm8", type="f16", q="e4m3", M=37, N=5003, K=4099, squares=True),
        # a square product, one tile or so per compute unit
        dict(name="gemm8-square", op="gemm8", type="bf16", q="e4m3", M=4096, N=4096, K=4096, squares=True),
        # the feed-forward product of a training step
        dict(name="gemm8-ffn", op="gemm8", type="bf16", q="e4m3", M=16384, N=28672, K=8192, squares=True),
        # a weight's gradient: both operands scaled along their rows, gradients of the wide-range type
        dict(name="gemm8-weight-grad", op="gemm8", type="f32", q="e5m2", M=8192, N=8192, K=16384, squares=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "norm_grad", "quant", "gemm8", "gemm8"])
    limit = [work(c) for c in listed() if c["op"] == op or (op == "norm" and c["op"] == "norm8")]
    most_bytes, most_flops = max(x["bytes"] for x in limit), max(x["flops"] for x in limit)
    while True:
        if op == "gemm8":
            c = dict(op=op, type=rng.choice(["bf16", "bf16", "f16", "f32"]), q=rng.choice(["e4m3", "e4m3", "e5m2"]),
                     M=_log(rng, 1, 16384), N=_log(rng, 64, 28672), K=_log(rng, 64, 28672),
                     squares=rng.random() < 0.67)
            widths = ("N", "K")
        else:
            c = dict(op=op, type=rng.choice(["bf16", "f16", "f32"]), N=_log(rng, 1, 65536), D=_log(rng, 32, 16384),
                     pad=rng.choice([0, 0, 8, 3]))
            if op.startswith("norm"):
                c["residual"] = rng.random() < 0.67
            else:
                c["squares"], c["forms"] = rng.random() < 0.5, rng.choice(["plain", "transposed", "both"])
            if op in ("norm8", "quant"):
                c["q"] = rng.choice(["e4m3", "e4m3", "e5m2"])
            widths = ("D",)
        if rng.random() < 0.5:  # half of the widths as programs choose them
            for k in widths:
                c[k] = max(64, c[k] // 64 * 64)
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    e = BYTES[case["type"]]
    if case["op"] == "gemm8":  # both operands and their scales read, C written
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * _blocks(K) * (M + (_blocks(N) if case["squares"] else N))
        return {"bytes": (M + N) * K + M * N * e + scales, "flops": 2 * M * N * K}
    N, D = case["N"], case["D"]
    n = N * D
    if case["op"] == "quant":  # x read once, each form and its scales written
        forms = 2 if case["forms"] == "both" else 1
        scales = 4 * _blocks(D) * (_blocks(N) if case["squares"] else N) * forms
        return {"bytes": n * (e + forms) + scales, "flops": 3 * n}
    extra = int(case["residual"])
    if case["op"] == "norm_grad":  # dy, h and the residual's gradient read, dx written; the weight and its gradient
        return {"bytes": n * e * (3 + extra) + 4 * N + 8 * D, "flops": 10 * n}
    out = 1 + 4 / BLOCK if case["op"] == "norm8" else e  # x and the residual read, their sum and y written
    return {"bytes": int(n * (e + 2 * e * extra + out)) + 4 * N + 4 * D, "flops": 7 * n}


def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(ord(ch) for ch in case["op"]) + 7 * case["N"])
    return g


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _activations(g, N, D):
    """Rows of different size, and a few columns that stand far out."""
    x = _normal(g, (N, D)) * torch.exp(_normal(g, (N, 1), 0.5))
    far = torch.rand(D, generator=g, device="cuda") < 0.004
    return x * torch.where(far, 20.0, 1.0)


def _rows(t, pad, dtype):
    """The same values in rows of the width + pad elements."""
    out = torch.empty((t.shape[0], t.shape[1] + pad), dtype=dtype, device=t.device)[:, :t.shape[1]]
    return out.copy_(t)


def _padded(t, rows):
    """t [r][d] with zeros up to whole blocks, as [blocks of rows][rows][blocks][128]."""
    r, d = t.shape
    t = torch.nn.functional.pad(t, (0, _blocks(d) * BLOCK - d, 0, -(-r // rows) * rows - r))
    return t.view(-1, rows, _blocks(d), BLOCK)


def _quantise(x, q, squares):
    """(q, scale) of fp32 x [N][D]: scales [N][blocks of D], or [blocks of N][blocks of D] for squares."""
    N, D = x.shape
    v = _padded(x, BLOCK if squares else 1)
    amax = v.abs().amax((1, 3))
    scale = (amax / LARGEST[q]).clamp_min(SMALLEST_SCALE)
    v = (v * (1.0 / scale)[:, None, :, None]).to(DTYPES[q])
    return v.reshape(-1, _blocks(D) * BLOCK)[:N, :D], scale


def _operand(x, q, squares):
    """An operand of the product as it is kept: rows 16 bytes aligned, row scales one block after the other."""
    v, scale = _quantise(x, q, squares)
    keep = torch.empty((v.shape[0], -(-v.shape[1] // 16) * 16), dtype=v.dtype, device=v.device)[:, :v.shape[1]]
    keep.copy_(v)
    return keep, scale if squares else scale.t().contiguous().t()


def prepare(case, seed):
    g = _generator(case, seed)
    s = {k: case[k] for k in ("op", "type", "q", "squares", "forms") if k in case}
    dt = DTYPES[case["type"]]
    if case["op"] == "gemm8":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(g, M, K) if case["q"] == "e4m3" else _normal(g, (M, K), 1e-4) * torch.exp(_normal(g, (M, 1)))
        s["a"], s["sa"] = _operand(x, case["q"], False)
        w = _normal(g, (N, K), 1 / math.sqrt(K)) if case["squares"] else _activations(g, N, K) / math.sqrt(K)
        s["b"], s["sb"] = _operand(w, "e4m3", case["squares"])
        return s
    N, D, pad = case["N"], case["D"], case["pad"]
    if case["op"] == "quant":
        x = _normal(g, (N, D), 1 / math.sqrt(D)) if case["squares"] else _activations(g, N, D)
        s["x"] = _rows(x, pad, dt)
        return s
    s["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
    s["x"] = _rows(_activations(g, N, D), pad, dt)
    s["residual"] = _rows(_activations(g, N, D), pad, dt) if case["residual"] else None
    if case["op"] == "norm_grad":  # x is then the sum that the norm saw, the residual the gradient of its other path
        s["dy"] = _rows(_normal(g, (N, D)), pad, dt)
        s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
    return s


def _plain(s):
    if s["op"] == "gemm8":
        a = _padded(s["a"].float(), 1) * s["sa"][:, None, :, None]
        b = _padded(s["b"].float(), BLOCK if s["squares"] else 1) * s["sb"][:, None, :, None]
        a, b = a.view(a.shape[0], -1), b.view(-1, a.shape[2] * BLOCK)[: s["b"].shape[0]]
        return (a @ b.t()).to(DTYPES[s["type"]])
    if s["op"] == "quant":
        out = {}
        if s["forms"] != "transposed":
            out["q"], out["scale"] = _quantise(s["x"].float(), s["q"], s["squares"])
        if s["forms"] != "plain":
            out["qt"], out["scale_t"] = _quantise(s["x"].float().t(), s["q"], s["squares"])
        return out
    t = s["x"].dtype
    if s["op"] == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        n = s["x"].float() * rstd
        h = dy * s["gamma"].float()
        dx = (h - n * (h * n).mean(1, keepdim=True)) * rstd
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return {"dx": dx.to(t), "dgamma": (dy * n).sum(0).to(t)}
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["h"] = (h + s["residual"].float()).to(t)
        h = out["h"].float()
    rstd = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * rstd.unsqueeze(1) * s["gamma"].float()
    out["rstd"] = rstd
    if s["op"] == "norm":
        out["y"] = y.to(t)
    else:
        out["q"], out["scale"] = _quantise(y, s["q"], False)
    return out


def _own(s):
    import recsys_linear_layers_amd as ll
    if s["op"] == "gemm8":
        return ll.gemm8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=DTYPES[s["type"]])
    if s["op"] == "quant":
        q = DTYPES[s["q"]]
        if s["forms"] == "both":
            return dict(zip(("q", "scale", "qt", "scale_t"), ll.quant8_pair(s["x"], squares=s["squares"], dtype=q)))
        names = ("q", "scale") if s["forms"] == "plain" else ("qt", "scale_t")
        return dict(zip(names, ll.quant8(s["x"], squares=s["squares"], transpose=s["forms"] == "transposed", dtype=q)))
    if s["op"] == "norm_grad":
        dx, dgamma = ll.rmsnorm_grad(s["dy"], s["x"], s["rstd"], s["gamma"], dh=s["residual"])
        return {"dx": dx, "dgamma": dgamma}
    if s["op"] == "norm":
        y, h, rstd = ll.rmsnorm(s["x"], s["gamma"], residual=s["residual"], eps=EPS)
        out = {"y": y, "rstd": rstd}
    else:
        q, scale, h, rstd = ll.rmsnorm8(s["x"], s["gamma"], residual=s["residual"], eps=EPS, dtype=DTYPES[s["q"]])
        out = {"q": q, "scale": scale, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    return out


def run(state):
    return _own(state) if own else _plain(state)


def _to_8_bits(v, q):
    """64-bit values rounded to the nearest value of the 8-bit type, ties to the even one."""
    digits, smallest = (3, -6) if q == "e4m3" else (2, -14)
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 1).clamp_min(smallest) - digits)
    return torch.round(v / step) * step


def _exact_quant(x, q, squares):
    """x in 64 bits, a block of 128 columns at a time."""
    N, D = x.shape
    out = torch.empty((N, D), dtype=torch.float64, device="cuda")
    of_row = torch.arange(N, device="cuda") // (BLOCK if squares else 1)
    scales = []
    for c in range(0, D, BLOCK):
        v = x[:, c:c + BLOCK]
        top = torch.zeros(int(of_row[-1]) + 1, dtype=torch.float64, device="cuda")
        top.scatter_reduce_(0, of_row, v.abs().max(1).values, "amax")
        top = torch.maximum(top / LARGEST[q], torch.full_like(top, SMALLEST_SCALE))
        out[:, c:c + BLOCK] = _to_8_bits(v / top[of_row, None], q)
        scales.append(top)
    return out, torch.stack(scales, 1)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "gemm8":
        c = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
        of_row = torch.arange(case["N"], device="cuda") // (BLOCK if case["squares"] else 1)
        for b, k in enumerate(range(0, case["K"], BLOCK)):
            left = s["a"][:, k:k + BLOCK].double() * s["sa"][:, b, None].double()
            right = s["b"][:, k:k + BLOCK].double() * s["sb"][of_row, b][:, None].double()
            c.addmm_(left, right.T)
        return c
    if case["op"] == "quant":
        out = {}
        if case["forms"] in ("plain", "both"):
            out["q"], out["scale"] = _exact_quant(s["x"].double(), case["q"], case["squares"])
        if case["forms"] in ("transposed", "both"):
            out["qt"], out["scale_t"] = _exact_quant(s["x"].double().T, case["q"], case["squares"])
        return out
    x, gamma = s["x"].double(), s["gamma"].double()
    if case["op"] == "norm_grad":
        normed = x * s["rstd"].double()[:, None]
        dy = s["dy"].double()
        along = (dy * normed * gamma).mean(1)
        dx = s["rstd"].double()[:, None] * (dy * gamma - normed * along[:, None])
        if s["residual"] is not None:
            dx += s["residual"].double()
        return {"dx": dx, "dgamma": torch.linalg.vecdot(dy, normed, dim=0)}
    out = {}
    if s["residual"] is not None:  # the norm is that of the sum as it is stored
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
        out["h"] = x
    out["rstd"] = 1.0 / torch.sqrt(x.pow(2).sum(1) / case["D"] + EPS)
    y = x * out["rstd"][:, None] * gamma
    if case["op"] == "norm":
        out["y"] = y
    else:
        out["q"], out["scale"] = _exact_quant(y, case["q"], False)
    return out
