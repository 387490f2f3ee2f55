"""What the embedding and layer norm entry points refuse, checked on the host
before any device is asked for (no GPU needed)."""
import ctypes

import pytest

P = 4096      # pointers stand far enough apart for these sizes; nothing reads them
Q = 1 << 30
R = 1 << 31


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


def _status(fn, desc, *args):
    ll = _ll()
    return ll.ll_status_string(fn(ctypes.byref(desc), *args))


def _embed(**kw):
    ll = _ll()
    base = dict(V=10, T=4, D=16, stride_table=16, stride_out=16, type=ll.LL_BF16, scale=1.0)
    base.update(kw)
    return ll.EmbedDesc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(V=-1), "LL_ERR_INVALID_ARG"), (dict(T=-1), "LL_ERR_INVALID_ARG"), (dict(D=-1), "LL_ERR_INVALID_ARG"),
    (dict(stride_table=15), "LL_ERR_INVALID_ARG"), (dict(stride_out=15), "LL_ERR_INVALID_ARG"),
    (dict(type=3), "LL_ERR_UNSUPPORTED"), (dict(V=1 << 31), "LL_ERR_UNSUPPORTED"),
    (dict(T=1 << 31), "LL_ERR_UNSUPPORTED"), (dict(stride_out=1 << 60), "LL_ERR_UNSUPPORTED"),
    (dict(scale=float("nan")), "LL_ERR_INVALID_ARG"), (dict(scale=float("inf")), "LL_ERR_INVALID_ARG"),
])
def test_embed_descriptions(kw, expect):
    assert _status(_ll()._lib.embed_run, _embed(**kw), P, Q, R, None) == expect


def test_embed_pointers():
    ll = _ll()
    run = ll._lib.embed_run
    assert run(None, P, Q, R, None) == ll.LL_ERR_INVALID_ARG
    for args in ((None, Q, R), (P, None, R), (P, Q, None), (P + 1, Q, R), (P, Q + 4, R), (P, Q, R + 1),
                 (P, Q, P), (P, Q, Q), (P, R + 8, R)):
        assert _status(run, _embed(), *args, None) == "LL_ERR_INVALID_ARG", args
    for kw in (dict(T=0), dict(D=0)):  # nothing to do: no pointer, no device
        assert _status(run, _embed(**kw), None, None, None, None) == "LL_OK"


def _embed_grad(**kw):
    ll = _ll()
    base = dict(V=10, T=4, D=16, stride_dout=16, stride_dtable=16, padding_id=-1, type=ll.LL_BF16, scale=1.0, flags=0)
    base.update(kw)
    return ll.EmbedGradDesc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(V=-1), "LL_ERR_INVALID_ARG"), (dict(stride_dout=3), "LL_ERR_INVALID_ARG"),
    (dict(padding_id=-2), "LL_ERR_INVALID_ARG"), (dict(flags=2), "LL_ERR_INVALID_ARG"),
    (dict(type=9), "LL_ERR_UNSUPPORTED"), (dict(scale=float("nan")), "LL_ERR_INVALID_ARG"),
])
def test_embed_grad_descriptions(kw, expect):
    ll = _ll()
    n = ctypes.c_size_t()
    assert _status(ll._lib.embed_grad_workspace_size, _embed_grad(**kw), ctypes.byref(n)) == expect
    assert _status(ll._lib.embed_grad_run, _embed_grad(**kw), P, Q, R, None, 0, None) == expect


def test_embed_grad_pointers_and_workspace():
    ll = _ll()
    run = ll._lib.embed_grad_run
    assert ll.embed_grad_workspace_size(_embed_grad(T=512)) == 0
    big = _embed_grad(T=513)
    need = ll.embed_grad_workspace_size(big)
    assert need > 0
    assert _status(run, big, P, Q, R, None, 0, None) == "LL_ERR_WORKSPACE"
    assert _status(run, big, P, Q, R, None, need, None) == "LL_ERR_WORKSPACE"
    assert _status(run, big, P, Q, R, 3 << 30, need - 1, None) == "LL_ERR_WORKSPACE"
    assert _status(run, big, P, Q, R, (3 << 30) + 128, need, None) == "LL_ERR_WORKSPACE"
    assert _status(run, big, P, Q, R, R, need, None) == "LL_ERR_INVALID_ARG"  # dtable inside the workspace
    for args in ((None, Q, R), (P, None, R), (P, Q, None), (P + 4, Q, R), (P, Q + 1, R), (P, Q, R + 1), (P, Q, Q)):
        assert _status(run, _embed_grad(), *args, None, 0, None) == "LL_ERR_INVALID_ARG", args
    assert _status(run, _embed_grad(V=0), None, None, None, None, 0, None) == "LL_OK"
    assert ll._lib.embed_grad_workspace_size(ctypes.byref(big), None) == ll.LL_ERR_INVALID_ARG
    assert ll._lib.embed_grad_workspace_size(None, None) == ll.LL_ERR_INVALID_ARG


def _norm(**kw):
    ll = _ll()
    base = dict(N=4, D=16, stride_x=16, stride_y=16, type=ll.LL_BF16, param_type=ll.LL_BF16, eps=1e-5)
    base.update(kw)
    return ll.LayernormDesc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "LL_ERR_INVALID_ARG"), (dict(D=-1), "LL_ERR_INVALID_ARG"), (dict(stride_x=15), "LL_ERR_INVALID_ARG"),
    (dict(stride_y=0), "LL_ERR_INVALID_ARG"), (dict(eps=-1.0), "LL_ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "LL_ERR_INVALID_ARG"), (dict(type=5), "LL_ERR_UNSUPPORTED"),
    (dict(param_type=2), "LL_ERR_UNSUPPORTED"), (dict(type=1, param_type=0), "LL_ERR_UNSUPPORTED"),
    (dict(D=1 << 31, stride_x=1 << 31, stride_y=1 << 31), "LL_ERR_UNSUPPORTED"),
])
def test_layernorm_descriptions(kw, expect):
    assert _status(_ll()._lib.layernorm_run, _norm(**kw), P, None, None, R, None, None, None) == expect


def test_layernorm_pointers():
    ll = _ll()
    run = ll._lib.layernorm_run
    assert run(None, P, None, None, R, None, None, None) == ll.LL_ERR_INVALID_ARG
    G, M = 3 << 30, 5 << 30
    for args in ((None, None, None, R, None, None), (P, None, None, None, None, None), (P + 1, None, None, R, None, None),
                 (P, G + 1, None, R, None, None), (P, None, None, P + 32, None, None), (P, G, None, G, None, None),
                 (P, None, None, R, M + 2, None), (P, None, None, R, M, M), (P, None, None, R, R, None),
                 (P, None, None, R, P, None)):
        assert _status(run, _norm(), *args, None) == "LL_ERR_INVALID_ARG", args
    # in place needs the same stride
    assert _status(run, _norm(stride_y=24), P, None, None, P, None, None, None) == "LL_ERR_INVALID_ARG"
    assert _status(run, _norm(N=0), None, None, None, None, None, None, None) == "LL_OK"


def _norm_grad(**kw):
    ll = _ll()
    base = dict(N=4, D=16, stride_dy=16, stride_x=16, stride_dx=16, type=ll.LL_F16, param_type=ll.LL_F32)
    base.update(kw)
    return ll.LayernormGradDesc(**base)


def test_layernorm_grad_refusals():
    ll = _ll()
    run, size = ll._lib.layernorm_grad_run, ll._lib.layernorm_grad_workspace_size
    n = ctypes.c_size_t()
    for kw, expect in ((dict(N=-1), "LL_ERR_INVALID_ARG"), (dict(stride_dy=8), "LL_ERR_INVALID_ARG"),
                       (dict(stride_dx=8), "LL_ERR_INVALID_ARG"), (dict(type=4), "LL_ERR_UNSUPPORTED"),
                       (dict(param_type=0), "LL_ERR_UNSUPPORTED")):
        assert _status(size, _norm_grad(**kw), ctypes.byref(n)) == expect, kw
    d = _norm_grad()
    need = ll.layernorm_grad_workspace_size(d)
    W, S, T, DX, DG, DB = 3 << 30, 5 << 30, 6 << 30, 7 << 30, 8 << 30, 9 << 30
    args = [P, Q, None, S, T, DX, DG, DB]
    assert _status(run, d, *args, None, 0, None) == "LL_ERR_WORKSPACE"
    assert _status(run, d, *args, W, need - 1, None) == "LL_ERR_WORKSPACE"
    assert _status(run, d, *args, W + 64, need, None) == "LL_ERR_WORKSPACE"
    for i, bad in ((0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (7, None), (5, P), (5, Q), (6, S),
                   (7, DG), (5, W), (0, P + 1), (6, DG + 2)):
        a = list(args)
        a[i] = bad
        assert _status(run, d, *a, W, need, None) == "LL_ERR_INVALID_ARG", (i, bad)
    assert _status(run, _norm_grad(N=0), None, None, None, None, None, None, None, None, None, 0, None) == "LL_OK"


def test_python_checks():
    torch = pytest.importorskip("torch")
    ll = _ll()
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ll.embedding(x, ids.int()), lambda: ll.embedding(x.t(), ids), lambda: ll.embedding(x[0], ids),
                 lambda: ll.embedding(x, ids, out=torch.zeros(4, 9)), lambda: ll.embedding(x.double(), ids),
                 lambda: ll.embedding(x, ids), lambda: ll.layernorm(x), lambda: ll.embedding_grad(ids, x, 5),  # on the host
                 lambda: ll.embedding_grad(ids, x[:3], 5), lambda: ll.embedding_grad(ids, x, 5, accumulate=True),
                 lambda: ll.embedding_grad(ids, x, 5, padding_idx=-1),
                 lambda: ll.embedding_grad(ids, x, 5, out=torch.zeros(5, 8, dtype=torch.float16)),
                 lambda: ll.layernorm(x, torch.ones(7)), lambda: ll.layernorm(x, torch.ones(8).half()),
                 lambda: ll.layernorm(x.bfloat16(), torch.ones(8), torch.ones(8).bfloat16()),
                 lambda: ll.layernorm(x, out=torch.zeros(4, 8).half()),
                 lambda: ll.layernorm_grad(x, x.half(), torch.ones(4), torch.ones(4)),
                 lambda: ll.layernorm_grad(x, x, torch.ones(3), torch.ones(4))):
        with pytest.raises((ValueError, TypeError)):
            call()


def _xent(**kw):
    ll = _ll()
    base = dict(N=4, V=100, D=16, stride_x=16, stride_w=16, stride_dx=16, stride_dw=16, ignore_index=-100,
                piece_bytes=0, type=ll.LL_BF16, dx_type=ll.LL_BF16, dw_type=ll.LL_F32, flags=3)
    base.update(kw)
    return ll.XentDesc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "LL_ERR_INVALID_ARG"), (dict(V=0), "LL_ERR_INVALID_ARG"), (dict(D=0), "LL_ERR_INVALID_ARG"),
    (dict(stride_x=15), "LL_ERR_INVALID_ARG"), (dict(stride_w=15), "LL_ERR_INVALID_ARG"),
    (dict(stride_dx=15), "LL_ERR_INVALID_ARG"), (dict(stride_dw=15), "LL_ERR_INVALID_ARG"),
    (dict(piece_bytes=-1), "LL_ERR_INVALID_ARG"), (dict(flags=8), "LL_ERR_INVALID_ARG"),
    (dict(type=1), "LL_ERR_UNSUPPORTED"), (dict(dx_type=2), "LL_ERR_UNSUPPORTED"),
    (dict(dw_type=2), "LL_ERR_UNSUPPORTED"), (dict(V=1 << 30), "LL_ERR_UNSUPPORTED"),
    (dict(D=1 << 20, stride_x=1 << 20, stride_w=1 << 20, stride_dx=1 << 20, stride_dw=1 << 20), "LL_ERR_UNSUPPORTED"),
    (dict(stride_x=1 << 28), "LL_ERR_UNSUPPORTED"),
])
def test_xent_descriptions(kw, expect):
    ll = _ll()
    h = ctypes.c_void_p()
    assert ll.ll_status_string(ll._lib.xent_plan_create(ctypes.byref(h), ctypes.byref(_xent(**kw)))) == expect
    assert not h.value


def test_xent_null_arguments():
    ll = _ll()
    h = ctypes.c_void_p()
    n = ctypes.c_size_t()
    assert ll._lib.xent_plan_create(None, ctypes.byref(_xent())) == ll.LL_ERR_INVALID_ARG
    assert ll._lib.xent_plan_create(ctypes.byref(h), None) == ll.LL_ERR_INVALID_ARG
    assert ll._lib.xent_plan_workspace_size(None, ctypes.byref(n)) == ll.LL_ERR_INVALID_ARG
    assert ll._lib.xent_plan_describe(None, None, 0) == ll.LL_ERR_INVALID_ARG
    assert ll._lib.xent_run(None, P, Q, R, None, P, None, None, None, None, 0, None) == ll.LL_ERR_INVALID_ARG
    assert ll._lib.xent_plan_destroy(None) == ll.LL_OK


@pytest.mark.gpu
def test_xent_run_refusals():
    """These need a plan, which needs a device; every call is refused on the host.
    The buffers are real, and far larger than the call needs."""
    import torch
    ll = _ll()
    h = ll.xent_plan_create(_xent())
    try:
        need = ll.xent_plan_workspace_size(h)
        run = ll._lib.xent_run
        room = 1 << 20
        assert need < room // 2
        buf = torch.zeros(9 * room, dtype=torch.uint8, device="cuda")
        X, W, T, G, L, E, DX, DW, WS = [buf.data_ptr() + i * room for i in range(9)]
        good = [X, W, T, G, L, E, DX, DW, WS]

        def status(args, ws_bytes=need):
            return ll.ll_status_string(run(h, *args, ws_bytes, None))

        assert status(good, need - 1) == "LL_ERR_WORKSPACE"
        for i, bad, want in ((0, None, "INVALID_ARG"), (1, None, "INVALID_ARG"), (2, None, "INVALID_ARG"),
                             (3, None, "INVALID_ARG"), (4, None, "INVALID_ARG"), (6, None, "INVALID_ARG"),
                             (7, None, "INVALID_ARG"), (8, None, "WORKSPACE"), (8, WS + 64, "WORKSPACE"),
                             (0, X + 1, "INVALID_ARG"), (1, W + 2, "INVALID_ARG"), (2, T + 4, "INVALID_ARG"),
                             (6, DX + 1, "INVALID_ARG"), (7, DW + 2, "INVALID_ARG"), (6, X, "INVALID_ARG"),
                             (7, W, "INVALID_ARG"), (4, E, "INVALID_ARG"), (5, G, "INVALID_ARG"),
                             (6, WS, "INVALID_ARG"), (7, DX, "INVALID_ARG")):
            a = list(good)
            a[i] = bad
            assert status(a) == "LL_ERR_" + want, (i, bad)
        assert status(good) == "LL_OK"
        torch.cuda.synchronize()
    finally:
        ll.xent_plan_destroy(h)
    with pytest.raises(ValueError):
        ll.vocab_xent(torch.zeros(2, 8).half(), torch.zeros(5, 9).half(), torch.zeros(2, dtype=torch.int64))
