"""Cases that measure the operators at the two ends of a model's linear layers:
the embedding lookup and its gradient by sorted tokens, layer norm and its
gradients, and the softmax cross entropy over a large vocabulary, taken in
pieces of the vocabulary, with its gradients.

``listed()`` and ``draw()`` give cases (dicts of plain values), ``prepare()``
the tensors a training or serving program has in hand, ``run()`` one pass.
Where the module's ``own`` is false ``run`` computes with elementary torch
operations in fp32; where it is true it calls recsys_linear_layers_amd.

Case keys: ``op`` (embed, embed_grad, norm, norm_grad, xent, xent_grad),
``type`` (of the tensors), and the sizes: ``T`` tokens, ``V`` rows of the table
(vocabulary), ``D`` width, ``N`` rows; ``pad``: extra elements between rows.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
PADDING = 0        # the id that pads ragged histories: looked up, but without a gradient
IGNORED = -100     # target of a row that has none
IGNORED_SHARE = 0.05


def listed():
    return [
        # one decode step of one sequence: the latency of a single row
        dict(name="embed-one-token", op="embed", type="bf16", T=1, V=131072, D=4096, scale=64.0),
        # the tokens of a training step of a wide model
        dict(name="embed-batch", op="embed", type="bf16", T=32768, V=131072, D=4096, scale=64.0),
        # fine-tuning on one short document: few tokens, odd width
        dict(name="embed-grad-few-odd", op="embed_grad", type="f16", T=300, V=8191, D=1001, scale=1.0),
        # the training step of embed-batch's kind: a few tokens take a large share of the positions
        dict(name="embed-grad-vocabulary", op="embed_grad", type="bf16", T=32768, V=65536, D=4096, scale=64.0),
        # an item table of a recommender: many narrow rows, most of them untouched by a batch
        dict(name="embed-grad-items", op="embed_grad", type="f32", T=262144, V=1000003, D=64, scale=1.0),
        # one decode step: the latency of a single wide row
        dict(name="norm-one-row", op="norm", type="bf16", N=1, D=8192, pad=0),
        # the activations in front of the 16384 x 8192 x 28672 feed-forward product
        dict(name="norm-batch", op="norm", type="bf16", N=16384, D=8192, pad=0),
        # and their gradient, with those of the weight and the bias
        dict(name="norm-grad-batch", op="norm_grad", type="bf16", N=16384, D=8192, pad=0),
        # odd sizes, rows at an odd distance, full precision
        dict(name="norm-grad-odd", op="norm_grad", type="f32", N=8191, D=5003, pad=3),
        # scoring one next token or item: the latency of one row over the vocabulary
        dict(name="xent-one-row", op="xent", type="bf16", N=1, V=50021, D=2048),
        # a small batch with odd sizes, loss and both gradients
        dict(name="xent-grad-odd", op="xent_grad", type="f16", N=777, V=32003, D=1000),
        # the head of a training step: loss and both gradients over a large vocabulary
        dict(name="xent-grad-batch", op="xent_grad", type="bf16", N=4096, V=131072, D=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _largest(op):
    """The most work of a listed case of this kind (forward and gradient alike)."""
    kind = op.split("_")[0]
    w = [work(c) for c in listed() if c["op"].split("_")[0] == kind]
    return max(x["bytes"] for x in w), max(x["flops"] for x in w)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "xent", "xent_grad"])
    most_bytes, most_flops = _largest(op)
    while True:
        if op.startswith("embed"):
            c = dict(op=op, type=rng.choice(["bf16", "f16", "f32"]), T=_log(rng, 1, 262144), V=_log(rng, 1000, 1000003),
                     D=_log(rng, 32, 8192), scale=rng.choice([1.0, 64.0, 0.7]))
            fits = c["V"] * c["D"] * BYTES[c["type"]] <= 1 << 30
        elif op.startswith("norm"):
            c = dict(op=op, type=rng.choice(["bf16", "f16", "f32"]), N=_log(rng, 1, 65536), D=_log(rng, 32, 16384),
                     pad=rng.choice([0, 0, 8, 3]))
            fits = True
        else:
            c = dict(op=op, type=rng.choice(["bf16", "bf16", "f16"]), N=_log(rng, 1, 16384), V=_log(rng, 1000, 262144),
                     D=_log(rng, 64, 8192))
            fits = c["V"] * c["D"] <= 131072 * 4096
        if rng.random() < 0.5:  # half of the widths as programs choose them
            c["D"] = max(64, c["D"] // 64 * 64)
        w = work(c)
        if c["D"] != 3072 and fits and w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


def work(case):
    e, D = BYTES[case["type"]], case["D"]
    if case["op"] == "embed":      # T rows read, T rows written
        n = case["T"] * D
        return {"bytes": 2 * n * e + 8 * case["T"], "flops": n}
    if case["op"] == "embed_grad":  # T rows read, the table's gradient written
        n = case["T"] * D
        return {"bytes": n * e + 8 * case["T"] + case["V"] * D * e, "flops": 2 * n}
    n = case["N"] * D
    if case["op"] == "norm":       # x read; y, mean and 1/deviation written; weight and bias read
        return {"bytes": 2 * n * e + 8 * case["N"] + 2 * D * e, "flops": 8 * n}
    if case["op"] == "norm_grad":  # x and dy read, dx written; the weight read, its and the bias' gradient written
        return {"bytes": 3 * n * e + 8 * case["N"] + 3 * D * e, "flops": 16 * n}
    live = 1.0 - (IGNORED_SHARE if case["N"] > 16 else 0.0)  # rows without a target need no product
    product = int(2 * n * case["V"] * live)
    read = (n + case["V"] * D) * e + 8 * case["N"] + 8 * case["N"]
    if case["op"] == "xent":
        return {"bytes": read, "flops": product}
    return {"bytes": read + (n + case["V"] * D) * e + 4 * case["N"], "flops": 3 * product}


def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(ord(ch) for ch in case["op"]) + 7 * case["D"])
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _ids(g, n, V):
    """Ids whose frequency falls as one over their rank (id 0, which pads, among the frequent ones)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(V)).long() - 1).clamp_(0, V - 1)


def _rows(g, N, D, pad, dtype, std=1.0):
    """[N][D] with rows D + pad elements apart."""
    return _normal(g, (N, D + pad), dtype, std)[:, :D]


def prepare(case, seed):
    g = _generator(case, seed)
    dt, D = DTYPES[case["type"]], case["D"]
    s = {"op": case["op"]}
    if case["op"] == "embed":
        s["table"] = _normal(g, (case["V"], D), dt, 0.02)
        s["ids"] = _ids(g, case["T"], case["V"])
        s["scale"] = case["scale"]
    elif case["op"] == "embed_grad":
        s["ids"] = _ids(g, case["T"], case["V"])
        if case["T"] == 1:
            s["ids"].clamp_(min=1)
        s["dout"] = _normal(g, (case["T"], D), dt)
        s["rows"], s["scale"] = case["V"], case["scale"]
    elif case["op"].startswith("norm"):
        offset = torch.randn((case["N"], 1), generator=g, device="cuda")
        s["x"] = _rows(g, case["N"], D, case["pad"], dt)
        s["x"] += offset.to(dt)
        s["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        if case["op"] == "norm":
            s["beta"] = _normal(g, (D,), dt, 0.1)
        else:
            s["dy"] = _rows(g, case["N"], D, case["pad"], dt)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS).float()
    else:
        s["x"] = _normal(g, (case["N"], D), dt)
        s["w"] = _normal(g, (case["V"], D), dt, 1.5 / math.sqrt(D))
        s["target"] = _ids(g, case["N"], case["V"])
        if case["N"] > 16:
            s["target"][torch.rand(case["N"], generator=g, device="cuda") < IGNORED_SHARE] = IGNORED
        if case["op"] == "xent_grad":
            s["dloss"] = torch.rand(case["N"], generator=g, device="cuda") + 0.5
    return s


def _plain(s):
    if s["op"] == "embed":
        return (s["table"][s["ids"]].float() * s["scale"]).to(s["table"].dtype)
    if s["op"] == "embed_grad":
        d = s["dout"].float() * (s["ids"] != PADDING).unsqueeze(1) * s["scale"]
        return torch.zeros((s["rows"], d.shape[1]), device="cuda").index_add_(0, s["ids"], d).to(s["dout"].dtype)
    if s["op"] == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        xc = x - mean.unsqueeze(1)
        rstd = torch.rsqrt((xc * xc).mean(1) + EPS)
        y = xc * rstd.unsqueeze(1) * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if s["op"] == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        xhat = (s["x"].float() - s["mean"].unsqueeze(1)) * rstd
        h = dy * s["gamma"].float()
        dx = (h - h.mean(1, keepdim=True) - xhat * (h * xhat).mean(1, keepdim=True)) * rstd
        t = s["x"].dtype
        return {"dx": dx.to(t), "dgamma": (dy * xhat).sum(0).to(t), "dbeta": dy.sum(0).to(t)}
    live = s["target"] != IGNORED
    x = torch.where(live.unsqueeze(1), s["x"].float(), 0.0)
    w = s["w"].float()
    z = x @ w.t()
    m = z.amax(1)
    at = torch.where(live, s["target"], 0).unsqueeze(1)
    zt = z.gather(1, at).squeeze(1)
    e = torch.exp(z.sub_(m.unsqueeze(1)))
    total = e.sum(1)
    lse = torch.where(live, m + torch.log(total), 0.0)
    loss = torch.where(live, lse - zt, 0.0)
    if s["op"] == "xent":
        return {"loss": loss, "lse": lse}
    g = torch.where(live, s["dloss"], 0.0)
    dz = e.mul_((g / total).unsqueeze(1)).scatter_add_(1, at, -g.unsqueeze(1))
    return {"loss": loss, "lse": lse, "dx": (dz @ w).to(s["x"].dtype), "dw": (dz.t() @ x).to(s["w"].dtype)}


def _own(s):
    import recsys_linear_layers_amd as ll
    if s["op"] == "embed":
        return ll.embedding(s["table"], s["ids"], scale=s["scale"])
    if s["op"] == "embed_grad":
        return ll.embedding_grad(s["ids"], s["dout"], s["rows"], scale=s["scale"], padding_idx=PADDING)
    if s["op"] == "norm":
        y, mean, rstd = ll.layernorm(s["x"], s["gamma"], s["beta"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if s["op"] == "norm_grad":
        dx, dgamma, dbeta = ll.layernorm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if s["op"] == "xent":
        loss, lse = ll.vocab_xent(s["x"], s["w"], s["target"], ignore_index=IGNORED)
        return {"loss": loss, "lse": lse}
    loss, lse, dx, dw = ll.vocab_xent_grad(s["x"], s["w"], s["target"], s["dloss"], ignore_index=IGNORED)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    s = prepare(case, seed)
    D = case["D"]
    if case["op"] == "embed":
        return torch.index_select(s["table"], 0, s["ids"]).double() * s["scale"]
    if case["op"] == "embed_grad":
        out = torch.zeros((case["V"], D), dtype=torch.float64, device="cuda")
        keep = torch.nonzero(s["ids"] != PADDING).squeeze(1)
        for part in keep.split(1 << 14):
            out.index_add_(0, s["ids"][part], s["dout"][part].double())
        return out * s["scale"]
    if case["op"] == "norm":
        y = torch.empty((case["N"], D), dtype=torch.float64, device="cuda")
        mean = torch.empty(case["N"], dtype=torch.float64, device="cuda")
        rstd = torch.empty_like(mean)
        for r in range(0, case["N"], 4096):
            b = slice(r, r + 4096)
            x = s["x"][b].double()
            var, mean[b] = torch.var_mean(x, 1, correction=0)
            rstd[b] = 1.0 / torch.sqrt(var + EPS)
            y[b] = (x - mean[b, None]) * rstd[b, None] * s["gamma"].double() + s["beta"].double()
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        dx = torch.empty((case["N"], D), dtype=torch.float64, device="cuda")
        dgamma = torch.zeros(D, dtype=torch.float64, device="cuda")
        dbeta = torch.zeros_like(dgamma)
        for r in range(0, case["N"], 4096):
            b = slice(r, r + 4096)
            dy, rs = s["dy"][b].double(), s["rstd"][b].double()[:, None]
            n = (s["x"][b].double() - s["mean"][b].double()[:, None]) * rs
            dgamma += (dy * n).sum(0)
            dbeta += dy.sum(0)
            u = dy * s["gamma"].double()
            dx[b] = rs * (u - (u.sum(1)[:, None] + n * (u * n).sum(1)[:, None]) / D)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    w = s["w"].double()
    loss = torch.zeros(case["N"], dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    grad = case["op"] == "xent_grad"
    if grad:
        dx = torch.zeros((case["N"], D), dtype=torch.float64, device="cuda")
        dw = torch.zeros((case["V"], D), dtype=torch.float64, device="cuda")
    live = torch.nonzero(s["target"] >= 0).squeeze(1)
    for part in live.split(512):
        x, t = s["x"][part].double(), s["target"][part]
        z = torch.mm(x, w.T)
        lse[part] = torch.logsumexp(z, 1)
        loss[part] = lse[part] - z[torch.arange(len(part), device="cuda"), t]
        if grad:
            p = torch.exp(z - lse[part][:, None])
            p[torch.arange(len(part), device="cuda"), t] -= 1.0
            p *= s["dloss"][part].double()[:, None]
            dx[part] = torch.mm(p, w)
            dw.addmm_(p.T, x)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw} if grad else {"loss": loss, "lse": lse}
