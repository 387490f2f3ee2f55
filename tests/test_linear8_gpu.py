"""The 8-bit linear layer's operators together, as a model uses them: a residual
block and its gradients, one token, captured graphs, other streams, threads."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


class Block:
    """s = x + r;  u = norm(s) W1^T;  y = s + relu(u) W2^T, products in 8 bits."""

    def __init__(self, width, hidden, seed):
        import torch
        import helpers8 as h
        ll = _ll()
        self.g = (1 + 0.1 * h.normal((width,), seed)).cuda().to(torch.bfloat16)
        self.w1 = h.normal((hidden, width), seed + 1, torch.bfloat16, width ** -0.5).cuda()
        self.w2 = h.normal((width, hidden), seed + 2, torch.bfloat16, hidden ** -0.5).cuda()
        self.q1, self.q2 = ll.quant8_pair(self.w1, squares=True), ll.quant8_pair(self.w2, squares=True)

    def forward(self, x, r):
        import torch
        ll = _ll()
        q, sc, s, rstd = ll.rmsnorm8(x, self.g, residual=r)
        u = ll.gemm8(q, sc, *self.q1[:2])
        a = torch.relu(u)
        a8 = ll.quant8_pair(a)
        return s + ll.gemm8(*a8[:2], *self.q2[:2]), (s, rstd, u, a8)

    def backward(self, dy, kept):
        import torch
        ll = _ll()
        s, rstd, u, a8 = kept
        d8 = ll.quant8_pair(dy)
        dw2 = ll.gemm8(*d8[2:], *a8[2:], out_dtype=torch.float32)
        du = ll.gemm8(*d8[:2], *self.q2[2:]) * (u > 0)
        d8 = ll.quant8_pair(du)
        n8t = ll.quant8(ll.rmsnorm(s, self.g)[0], transpose=True)
        dw1 = ll.gemm8(*d8[2:], *n8t, out_dtype=torch.float32)
        dn = ll.gemm8(*d8[:2], *self.q1[2:])
        ds, dg = ll.rmsnorm_grad(dn, s, rstd, self.g, dh=dy)
        return {"ds": ds, "dg": dg, "dw1": dw1, "dw2": dw2}


def _reference(b, x, r, dy):
    """In 64 bits on the host, from the same 16-bit weights, nothing quantised."""
    import torch
    x, r, dy = x.double().cpu(), r.double().cpu(), dy.double().cpu()
    g, w1, w2 = (t.double().cpu().requires_grad_() for t in (b.g, b.w1, b.w2))
    s = (x + r).requires_grad_()
    n = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * g
    y = s + torch.relu(n @ w1.T) @ w2.T
    (y * dy).sum().backward()
    return y.detach(), {"ds": s.grad, "dg": g.grad, "dw1": w1.grad, "dw2": w2.grad}


@pytest.mark.parametrize("rows,width,hidden", [(1, 256, 512), (3, 200, 264), (70, 384, 1000), (300, 520, 768),
                                               (1025, 1024, 2048)])
def test_block_and_gradients(rows, width, hidden):
    """A value quantised in e4m3 is off by at most 2^-4 of itself, evenly spread:
    2^-4 / sqrt(3) = 3.6% of a tensor's norm, 5.1% of a product of two.  The result
    passes two products beside an exact path, a gradient up to three in a row, and
    a relu that flips near 0: at most 3 * 5.1% of the norm, and 5% more."""
    import helpers8 as h
    import torch
    b = Block(width, hidden, rows)
    x, r, dy = (h.normal((rows, width), k, torch.bfloat16).cuda() for k in (11, 12, 13))
    y, kept = b.forward(x, r)
    got = b.backward(dy, kept)
    want_y, want = _reference(b, x, r, dy)
    err = (y.double().cpu() - want_y).norm() / want_y.norm()
    assert err < 0.10, err
    for k, v in want.items():
        err = (got[k].double().cpu() - v).norm() / v.norm()
        assert err < 0.20, (k, err.item())
        assert bool(torch.isfinite(got[k]).all())


def test_a_row_alone_is_the_row_among_others():
    """Serving a row by itself or in a batch: every 8-bit operand and scale is the
    same, so the results differ by the products' order of addition alone."""
    import helpers8 as h
    import torch
    ll = _ll()
    b = Block(1024, 2048, 5)
    x, r = h.normal((300, 1024), 1, torch.bfloat16).cuda(), h.normal((300, 1024), 2, torch.bfloat16).cuda()
    q, sc, s, rstd = ll.rmsnorm8(x, b.g, residual=r)
    q1, sc1, s1, rstd1 = ll.rmsnorm8(x[7:8], b.g, residual=r[7:8])
    assert torch.equal(q[7:8].view(torch.uint8), q1.view(torch.uint8))
    assert torch.equal(sc[7:8], sc1) and torch.equal(s[7:8], s1) and torch.equal(rstd[7:8], rstd1)
    all_, one = ll.gemm8(q, sc, *b.q1[:2], out_dtype=torch.float32), ll.gemm8(q1, sc1, *b.q1[:2], out_dtype=torch.float32)
    A = h.dequantise(q1, sc1, False).abs() @ h.dequantise(*b.q1[:2], True).abs().T
    assert bool(((all_[7:8] - one).cpu().double().abs() <= 2 * (256 + 8 + 67) * h.U * A).all())


def _calls(seed=0):
    """One call of each operator, small and large enough for every path: name, call, outputs."""
    import helpers8 as h
    import torch
    ll = _ll()
    e4 = torch.float8_e4m3fn
    out = []
    for rows, D in ((3, 300), (600, 1030), (2, 20000)):
        x, r, dy = (h.normal((rows, D), seed + k, torch.bfloat16).cuda() for k in (1, 2, 3))
        g = h.normal((D,), seed + 4, torch.bfloat16).cuda()
        rstd = torch.rand(rows, generator=torch.Generator().manual_seed(seed + 5)).cuda() + 0.5
        out += [(f"norm8 {rows}", lambda x=x, r=r, g=g: ll.rmsnorm8(x, g, residual=r)),
                (f"norm {rows}", lambda x=x, g=g: ll.rmsnorm(x, g)[::2]),  # without a residual, the sum is x itself
                (f"grad {rows}", lambda x=x, r=r, g=g, dy=dy, s=rstd: ll.rmsnorm_grad(dy, x, s, g, dh=r)),
                (f"quant {rows}", lambda x=x: ll.quant8_pair(x)), (f"squares {rows}", lambda x=x: ll.quant8_pair(x, squares=True))]
    for M, N, K in ((1, 500, 700), (16, 900, 3000), (40, 300, 5000), (64, 4000, 8192), (130, 260, 9000), (700, 1030, 520),
                    (1500, 2100, 400)):
        a, sa = ll.quant8(h.normal((M, K), seed + 6).cuda())
        b, sb = ll.quant8(h.normal((N, K), seed + 7).cuda(), squares=True)
        for c in (torch.bfloat16, torch.float32):
            out.append((f"gemm8 {M} {c}", lambda a=a, sa=sa, b=b, sb=sb, c=c: (ll.gemm8(a, sa, b, sb, out_dtype=c),)))
    return out


def _bytes(ts):
    import torch
    return [t.reshape(-1).clone().view(torch.uint8) for t in ts if t is not None]


def _same(a, b):
    import torch
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed():
    """Each call in a graph of its own, replayed with eager work between; then all
    graphs once more, the first after the last (none keeps what another wrote)."""
    import torch
    calls = _calls()
    eager = [_bytes(f()) for _, f in calls]
    torch.cuda.synchronize()
    graphs = []
    for (name, f), want in zip(calls, eager):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = f()
        graphs.append((name, g, outs, want))
        for _ in range(3):
            for t in outs:
                t.copy_(torch.full(t.shape, 0.5, device="cuda").to(t.dtype))
            g.replay()
            torch.cuda.synchronize()
            assert _same(_bytes(outs), want), name
            torch.randn(300, 300, device="cuda").sum()
            torch.cuda.synchronize()
    for name, g, outs, want in graphs + graphs[:3]:
        g.replay()
        torch.cuda.synchronize()
        assert _same(_bytes(outs), want), name


def test_two_graphs_at_once():
    """Two captured calls that need workspaces, replayed on two streams at the same time."""
    import torch
    calls = [c for c in _calls() if c[0].startswith(("gemm8 130", "gemm8 64", "gemm8 40", "grad 600"))]
    assert len(calls) == 7
    eager = [_bytes(f()) for _, f in calls]
    graphs = []
    for name, f in calls:
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = f()
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        torch.cuda.synchronize()
        for (g, _o), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (g, outs), want, (name, _f) in zip(graphs, eager, calls):
            assert _same(_bytes(outs), want), name


def test_on_other_streams_and_threads():
    """The calls on a stream of each of two threads, and on one stream by both."""
    import threading

    import torch
    calls = _calls(20)
    want = [_bytes(f()) for _, f in calls]
    torch.cuda.synchronize()
    for shared in (False, True):
        one = torch.cuda.Stream()
        wrong = []

        def work(stream):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    got = [f() for _, f in calls]
                    got = [_bytes(g) for g in got]
                    stream.synchronize()
                    wrong.extend(n for (n, _f), g, w in zip(calls, got, want) if not _same(g, w))

        threads = [threading.Thread(target=work, args=(one if shared else torch.cuda.Stream(),)) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join(60)
        torch.cuda.synchronize()
        assert not wrong, (shared, wrong)


def _example():
    spec = importlib.util.spec_from_file_location("next_item8", os.path.join(ROOT, "examples", "next_item.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("items,width,hidden,users,length", [(301, 64, 96, 9, 12), (2003, 200, 264, 70, 11)])
def test_example_in_8_bits_has_the_16_bit_gradients(items, width, hidden, users, length):
    """The same weights and batch with the middle's products in 16 and in 8 bits: a
    gradient passes at most three 8-bit products, 5.1% of its norm each (as above),
    and flips of the relu near 0."""
    import torch
    ex = _example()
    a, b = (ex.NextItem(items, width, hidden, seed=3, eight_bit=e) for e in (False, True))
    ids, target = ex.histories(users, length, items, seed=4)
    loss_a, grads_a = a.loss_and_grads(ids, target)
    loss_b, grads_b = b.loss_and_grads(ids, target)
    assert abs(loss_a.item() - loss_b.item()) <= 0.05 * loss_a.item()
    for k, g in grads_a.items():
        err = (grads_b[k].double() - g.double()).norm() / g.double().norm()
        assert err <= 0.20, (k, err.item())
        assert bool(torch.isfinite(grads_b[k]).all())
    b.update(grads_b)
