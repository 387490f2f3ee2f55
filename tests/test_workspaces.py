"""Scratch of the torch entry points: each call has its own.

The library lets go of the interpreter lock while it launches, so two threads'
launches on one stream may interleave; and a captured graph keeps the addresses
it saw.  On the host the C calls are stand-ins that meet inside and compare
the workspaces they were given; on the GPU the results are compared."""
import threading

import pytest


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


def _meet(monkeypatch, entry, ws_at, call):
    """The workspace addresses of two calls that are inside the C entry at the same time."""
    ll = _ll()
    inside = threading.Barrier(2, timeout=30)
    seen = []

    def stand_in(*args):
        seen.append((args[ws_at], args[ws_at + 1]))
        inside.wait()

    monkeypatch.setattr(ll, entry, stand_in)
    monkeypatch.setattr(ll, "_stream_of", lambda t: 0, raising=False)
    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert len(seen) == 2
    return seen


def test_two_threads_have_workspaces_of_their_own(monkeypatch):
    torch = pytest.importorskip("torch")
    ll = _ll()
    ids, dout = torch.zeros(600, dtype=torch.int64), torch.zeros(600, 8)
    x, s = torch.zeros(50, 16), torch.zeros(50)

    class Plan:
        handle, ws_bytes = 1, 4096

    monkeypatch.setattr(ll, "xent_plan_for", lambda *a, **k: Plan)
    h = torch.zeros(5, 8).half()
    for entry, ws_at, call in (
            ("embed_grad_run", 4, lambda: ll.embedding_grad(ids, dout, 50)),
            ("layernorm_grad_run", 9, lambda: ll.layernorm_grad(x, x, s, s)),
            ("xent_run", 9, lambda: ll.vocab_xent(h, h, torch.zeros(5, dtype=torch.int64)))):
        (a, n), (b, m) = _meet(monkeypatch, entry, ws_at, call)
        assert n == m > 0 and (a + n <= b or b + m <= a), entry


@pytest.mark.parametrize("stream", [None, 5])
def test_two_threads_that_run_one_gemm_plan_have_workspaces_of_their_own(monkeypatch, stream):
    torch = pytest.importorskip("torch")
    ll = _ll()

    class Stream:
        cuda_stream = 5

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    plan = ll.GemmPlan.__new__(ll.GemmPlan)  # a plan needs a device
    plan.desc, plan.handle, plan.ws_bytes, plan.device, plan._ws = ll.GemmDesc(), None, 4096, torch.device("cpu"), {}
    a = torch.zeros(4, 4)
    (p, n), (q, m) = _meet(monkeypatch, "gemm_run", 4, lambda: plan.run(a, a, a, stream))
    assert n == m == 4096 and (p + n <= q or q + m <= p)


def _calls(seed):
    """One call of each operator that takes a workspace, on inputs of its own."""
    import torch
    ll = _ll()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, 3000, (9000,), generator=g, device="cuda")
    dout = n(9000, 72)
    x, dy = n(2000, 384), n(2000, 384)
    y, mean, rstd = ll.layernorm(x)
    a, w = n(300, 200).bfloat16(), (n(5000, 200) / 14).bfloat16()
    target = torch.randint(0, 5000, (300,), generator=g, device="cuda")
    dloss = torch.rand(300, generator=g, device="cuda")
    return [lambda: (ll.embedding_grad(ids, dout, 3000),), lambda: ll.layernorm_grad(dy, x, mean, rstd),
            lambda: ll.vocab_xent_grad(a, w, target, dloss)]


def _same(got, want):
    import torch
    return all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.gpu
def test_two_threads_on_one_stream_get_the_serial_results():
    import torch
    work = [_calls(s) for s in (1, 2)]
    want = [[f() for f in calls] for calls in work]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2, timeout=30), []

    def run(k):
        try:
            start.wait()
            # the second thread takes the operators in another order
            got = [(i, work[k][i]()) for _ in range(40) for i in ((0, 1, 2) if k == 0 else (2, 0, 1))]
            wrong.extend((k, i) for i, out in got if not _same(out, want[k][i]))
        except Exception as e:  # a thread's own failure would be lost
            wrong.append((k, repr(e)))

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
    assert not wrong and not any(t.is_alive() for t in threads)


@pytest.mark.gpu
def test_two_threads_run_one_gemm_plan_on_one_stream():
    """Split K and packed operands: partials and copies in the workspace."""
    import torch
    ll = _ll()
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    pairs = [(torch.randn((64, 8193), generator=g, device="cuda").bfloat16(),
              torch.randn((8193, 320), generator=g, device="cuda").bfloat16()) for _ in range(2)]
    want = [ll.gemm(a, b, out_dtype=torch.float32) for a, b in pairs]
    plan = ll.plan_for(*pairs[0], want[0])
    assert plan.ws_bytes > 0
    torch.cuda.synchronize()
    start, got = threading.Barrier(2, timeout=30), [[], []]

    def run(k):
        start.wait()
        got[k] = [ll.gemm(*pairs[k], out_dtype=torch.float32) for _ in range(100)]

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
    assert all(len(got[k]) == 100 and all(torch.equal(c, want[k]) for c in got[k]) for k in range(2))


@pytest.mark.gpu
def test_a_captured_graph_outlives_larger_calls_on_its_stream():
    import torch
    ll = _ll()
    side = torch.cuda.Stream()
    for call in _calls(3):
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call()  # warm up, as a program does before it captures
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call()
        with torch.cuda.stream(side):  # a larger call of each operator on the same stream
            ids = torch.arange(100000, device="cuda")
            ll.embedding_grad(ids, torch.ones((100000, 72), device="cuda"), 100000)
            z = torch.ones((4000, 8192), device="cuda")
            ll.layernorm_grad(z, z, z[:, 0].contiguous(), z[:, 0].contiguous())
            h = torch.zeros((600, 200), dtype=torch.bfloat16, device="cuda")
            ll.vocab_xent_grad(h, torch.zeros((40000, 200), dtype=torch.bfloat16, device="cuda"), ids[:600],
                               torch.ones(600, device="cuda"))
            others = [torch.full((1 << k,), 7, dtype=torch.uint8, device="cuda") for k in range(10, 25) for _ in range(4)]
        torch.cuda.synchronize()
        for _ in range(3):
            for t in got:
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(got, want)
            assert all(bool((t == 7).all()) for t in others)


@pytest.mark.gpu
def test_two_graphs_replay_at_once():
    """Captured on one stream, replayed on two."""
    import torch
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = [_calls(s) for s in (4, 5)]
    for i in range(3):
        want = [work[k][i]() for k in range(2)]
        torch.cuda.synchronize()
        graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
        for k in range(2):
            with torch.cuda.graph(graphs[k]):
                got.append(work[k][i]())
        for _ in range(5):
            for out in got:
                for t in out:
                    t.fill_(float("nan"))
            torch.cuda.synchronize()
            for _ in range(4):
                for k in range(2):
                    with torch.cuda.stream(streams[k]):
                        graphs[k].replay()
            torch.cuda.synchronize()
            assert all(_same(got[k], want[k]) for k in range(2))
