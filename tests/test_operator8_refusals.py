"""What the 8-bit linear layers' entry points refuse, checked on the host before
any device is asked for (no GPU needed)."""
import ctypes

import pytest

P = 4096      # pointers stand far enough apart for these sizes; nothing reads them
Q, R, S, T = 1 << 30, 1 << 31, 3 << 30, 5 << 30


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


def _status(fn, desc, *args):
    ll = _ll()
    return ll.ll_status_string(fn(ctypes.byref(desc), *args))


# --- rmsnorm_run(desc, x, residual, gamma, h, y, scale, rstd, stream) ---------

def _norm(**kw):
    ll = _ll()
    base = dict(N=4, D=16, stride_x=16, stride_residual=16, stride_h=16, stride_y=16, stride_sn=1, stride_sb=4,
                type=ll.LL_BF16, param_type=ll.LL_BF16, y_type=ll.LL_BF16, eps=1e-6)
    base.update(kw)
    return ll.RmsnormDesc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "LL_ERR_INVALID_ARG"), (dict(D=-1), "LL_ERR_INVALID_ARG"), (dict(stride_x=15), "LL_ERR_INVALID_ARG"),
    (dict(stride_y=15), "LL_ERR_INVALID_ARG"), (dict(stride_residual=15), "LL_ERR_INVALID_ARG"),
    (dict(stride_h=0), "LL_ERR_INVALID_ARG"), (dict(eps=-1.0), "LL_ERR_INVALID_ARG"),
    (dict(eps=float("inf")), "LL_ERR_INVALID_ARG"), (dict(type=3), "LL_ERR_UNSUPPORTED"),
    (dict(param_type=2), "LL_ERR_UNSUPPORTED"), (dict(y_type=1), "LL_ERR_UNSUPPORTED"),
    (dict(y_type=5), "LL_ERR_UNSUPPORTED"), (dict(N=1 << 40), "LL_ERR_UNSUPPORTED"),
    (dict(y_type=3, stride_sn=0), "LL_ERR_INVALID_ARG"), (dict(y_type=3, stride_sb=-4), "LL_ERR_INVALID_ARG"),
    (dict(y_type=4, stride_sn=1 << 60), "LL_ERR_UNSUPPORTED"), (dict(stride_h=1 << 60), "LL_ERR_UNSUPPORTED"),
    (dict(D=1 << 30, stride_x=1 << 30, stride_y=1 << 30, stride_residual=1 << 30, stride_h=1 << 30),
     "LL_ERR_UNSUPPORTED"),
])
def test_rmsnorm_descriptions(kw, expect):
    assert _status(_ll()._lib.rmsnorm_run, _norm(**kw), P, Q, None, R, S, T, None, None) == expect


def test_rmsnorm_pointers():
    ll = _ll()
    run = ll._lib.rmsnorm_run
    assert run(None, P, None, None, None, S, None, None, None) == ll.LL_ERR_INVALID_ARG
    G = 7 << 30
    for args in ((None, None, None, None, S, None, None), (P, None, None, None, None, None, None),
                 (P, Q, None, None, S, None, None), (P, None, None, R, S, None, None),  # h and residual go together
                 (P + 1, None, None, None, S, None, None), (P, Q + 1, None, R, S, None, None),
                 (P, Q, None, R + 1, S, None, None), (P, None, G + 1, None, S, None, None),
                 (P, None, None, None, S, None, T + 2), (P, Q, None, R, R, None, None), (P, Q, None, R, Q, None, None),
                 (P, Q, None, P, P, None, None), (P, None, None, None, P + 32, None, None),
                 (P, Q, None, R, R + 64, None, None),
                 (P, None, G, None, G, None, None), (P, None, None, None, S, None, S), (P, None, None, None, S, None, P)):
        assert _status(run, _norm(), *args, None) == "LL_ERR_INVALID_ARG", args
    # 8-bit: a scale, apart from everything; y never over x
    for args in ((P, None, None, None, S, None, None), (P, None, None, None, S, T + 1, None),
                 (P, None, None, None, P, T, None), (P, None, None, None, S, S, None), (P, None, None, None, S, P, None),
                 (P, None, None, None, S, T, T)):
        assert _status(run, _norm(y_type=ll.LL_E4M3), *args, None) == "LL_ERR_INVALID_ARG", args
    # in place needs the same stride
    assert _status(run, _norm(stride_y=24), P, None, None, None, P, None, None, None) == "LL_ERR_INVALID_ARG"
    assert _status(run, _norm(stride_h=24), P, Q, None, Q, S, None, None, None) == "LL_ERR_INVALID_ARG"
    for kw in (dict(N=0), dict(D=0)):
        assert _status(run, _norm(**kw), *[None] * 7, None) == "LL_OK"


# --- rmsnorm_grad_run(desc, dy, h, gamma, rstd, dh, dx, dgamma, ws, bytes, stream)

def _grad(**kw):
    ll = _ll()
    base = dict(N=4, D=16, stride_dy=16, stride_h=16, stride_dh=16, stride_dx=16, type=ll.LL_BF16, param_type=ll.LL_BF16)
    base.update(kw)
    return ll.RmsnormGradDesc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "LL_ERR_INVALID_ARG"), (dict(stride_dy=15), "LL_ERR_INVALID_ARG"),
    (dict(stride_h=15), "LL_ERR_INVALID_ARG"), (dict(stride_dx=15), "LL_ERR_INVALID_ARG"),
    (dict(type=4), "LL_ERR_UNSUPPORTED"), (dict(param_type=2), "LL_ERR_UNSUPPORTED"),
])
def test_rmsnorm_grad_descriptions(kw, expect):
    ll = _ll()
    n = ctypes.c_size_t()
    assert _status(ll._lib.rmsnorm_grad_workspace_size, _grad(**kw), ctypes.byref(n)) == expect
    assert _status(ll._lib.rmsnorm_grad_run, _grad(**kw), P, Q, None, R, None, S, None, None, 0, None) == expect


def test_rmsnorm_grad_pointers_and_workspace():
    ll = _ll()
    run = ll._lib.rmsnorm_grad_run
    need = ll.rmsnorm_grad_workspace_size(_grad())
    assert need > 0
    W, G = 9 << 30, 7 << 30
    for args in ((None, Q, None, R, None, S, None), (P, None, None, R, None, S, None), (P, Q, None, None, None, S, None),
                 (P, Q, None, R, None, None, None), (P + 1, Q, None, R, None, S, None), (P, Q, None, R + 2, None, S, None),
                 (P, Q, None, R, T + 1, S, None), (P, Q, None, R, None, P, None), (P, Q, None, R, None, Q, None),
                 (P, Q, S, R, None, S, None), (P, Q, None, R, T, T + 2, None)):
        assert _status(run, _grad(), *args, None, 0, None) == "LL_ERR_INVALID_ARG", args
    assert _status(run, _grad(stride_dh=15), P, Q, None, R, T, S, None, None, 0, None) == "LL_ERR_INVALID_ARG"
    assert _status(run, _grad(stride_dh=24), P, Q, None, R, T, T, None, None, 0, None) == "LL_ERR_INVALID_ARG"
    for ws, n in ((None, 0), (None, need), (W, need - 1), (W + 128, need)):
        assert _status(run, _grad(), P, Q, None, R, None, S, G, ws, n, None) == "LL_ERR_WORKSPACE"
    for dgamma, ws in ((S, W), (P, W), (W, W), (G, S)):
        assert _status(run, _grad(), P, Q, None, R, None, S, dgamma, ws, need, None) == "LL_ERR_INVALID_ARG"
    assert _status(run, _grad(N=0), *[None] * 8, 0, None) == "LL_OK"
    assert ll._lib.rmsnorm_grad_workspace_size(ctypes.byref(_grad()), None) == ll.LL_ERR_INVALID_ARG


# --- quant8_run(desc, x, q, scale, qt, scale_t, stream) -----------------------

def _quant(**kw):
    ll = _ll()
    base = dict(N=4, D=20, stride_x=20, stride_q=32, stride_qt=16, stride_sn=1, stride_sb=4, stride_tn=1, stride_tb=20,
                type=ll.LL_BF16, q_type=ll.LL_E4M3, block=1)
    base.update(kw)
    return ll.Quant8Desc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), "LL_ERR_INVALID_ARG"), (dict(stride_x=19), "LL_ERR_INVALID_ARG"),
    (dict(stride_q=19), "LL_ERR_INVALID_ARG"), (dict(stride_qt=3), "LL_ERR_INVALID_ARG"),
    (dict(stride_sn=0), "LL_ERR_INVALID_ARG"), (dict(stride_tb=-1), "LL_ERR_INVALID_ARG"),
    (dict(block=64), "LL_ERR_INVALID_ARG"), (dict(type=3), "LL_ERR_UNSUPPORTED"), (dict(q_type=0), "LL_ERR_UNSUPPORTED"),
    (dict(D=1 << 30, stride_x=1 << 30, stride_q=1 << 30), "LL_ERR_UNSUPPORTED"),
    (dict(stride_qt=1 << 60), "LL_ERR_UNSUPPORTED"),
])
def test_quant8_descriptions(kw, expect):
    assert _status(_ll()._lib.quant8_run, _quant(**kw), P, Q, R, S, T, None) == expect


def test_quant8_pointers():
    ll = _ll()
    run = ll._lib.quant8_run
    assert run(None, P, Q, R, S, T, None) == ll.LL_ERR_INVALID_ARG
    for args in ((None, Q, R, S, T), (P, None, None, None, None), (P, Q, None, S, T), (P, None, R, S, T),
                 (P, Q, R, None, T), (P, Q, R, S, None), (P + 1, Q, R, S, T), (P, Q, R + 2, S, T), (P, Q, R, S, T + 1),
                 (P, P + 8, R, S, T), (P, Q, P, S, T), (P, Q, R, Q, T), (P, Q, R, S, R), (P, Q, Q, S, T)):
        assert _status(run, _quant(), *args, None) == "LL_ERR_INVALID_ARG", args
    for kw in (dict(N=0), dict(D=0)):
        assert _status(run, _quant(**kw), *[None] * 5, None) == "LL_OK"


# --- gemm8_run(desc, A, a_scale, B, b_scale, C, ws, bytes, stream) ------------

def _gemm(**kw):
    ll = _ll()
    base = dict(M=4, N=20, K=40, stride_a=48, stride_b=48, stride_c=20, stride_am=1, stride_ab=4, stride_bn=1,
                stride_bb=1, a_type=ll.LL_E4M3, b_type=ll.LL_E4M3, c_type=ll.LL_BF16, b_block=128)
    base.update(kw)
    return ll.Gemm8Desc(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), "LL_ERR_INVALID_ARG"), (dict(K=-1), "LL_ERR_INVALID_ARG"), (dict(stride_a=32), "LL_ERR_INVALID_ARG"),
    (dict(stride_b=56), "LL_ERR_INVALID_ARG"), (dict(stride_c=19), "LL_ERR_INVALID_ARG"),
    (dict(b_block=2), "LL_ERR_INVALID_ARG"), (dict(stride_am=0), "LL_ERR_INVALID_ARG"),
    (dict(stride_bb=0), "LL_ERR_INVALID_ARG"), (dict(a_type=0), "LL_ERR_UNSUPPORTED"),
    (dict(b_type=4), "LL_ERR_UNSUPPORTED"), (dict(c_type=3), "LL_ERR_UNSUPPORTED"), (dict(M=1 << 26), "LL_ERR_UNSUPPORTED"),
    (dict(N=1 << 26, stride_c=1 << 26), "LL_ERR_UNSUPPORTED"),
    (dict(M=1 << 25, N=1 << 25, stride_c=1 << 25), "LL_ERR_UNSUPPORTED"),
    (dict(K=1 << 22, stride_a=1 << 22, stride_b=1 << 22), "LL_ERR_UNSUPPORTED"),
    (dict(stride_a=1 << 22), "LL_ERR_UNSUPPORTED"), (dict(stride_am=1 << 20), "LL_ERR_UNSUPPORTED"),
    (dict(b_block=1, stride_bn=1 << 20), "LL_ERR_UNSUPPORTED"), (dict(stride_ab=1 << 60), "LL_ERR_UNSUPPORTED"),
])
def test_gemm8_descriptions(kw, expect):
    ll = _ll()
    n = ctypes.c_size_t()
    assert _status(ll._lib.gemm8_workspace_size, _gemm(**kw), ctypes.byref(n)) == expect
    assert _status(ll._lib.gemm8_describe, _gemm(**kw), ctypes.create_string_buffer(64), 64) == expect
    assert _status(ll._lib.gemm8_run, _gemm(**kw), P, Q, R, S, T, None, 0, None) == expect


def test_gemm8_pointers_and_workspace():
    ll = _ll()
    run = ll._lib.gemm8_run
    assert run(None, P, Q, R, S, T, None, 0, None) == ll.LL_ERR_INVALID_ARG
    for args in ((None, Q, R, S, T), (P, None, R, S, T), (P, Q, None, S, T), (P, Q, R, None, T), (P, Q, R, S, None),
                 (P + 8, Q, R, S, T), (P, Q, R + 8, S, T), (P, Q + 2, R, S, T), (P, Q, R, S, T + 1),
                 (P, Q, R, S, P), (P, Q, R, S, Q), (P, Q, R, S, R + 64), (P, Q, R, S, S)):
        assert _status(run, _gemm(), *args, None, 0, None) == "LL_ERR_INVALID_ARG", args
    for kw in (dict(M=0), dict(N=0)):
        assert _status(run, _gemm(**kw), *[None] * 6, 0, None) == "LL_OK"
    big = _gemm(M=128, N=256, K=100000, stride_a=100000, stride_b=100000, stride_c=256, stride_ab=128, stride_bb=2)
    need = ll.gemm8_workspace_size(big)
    assert need > 0 and "splits=" in ll.gemm8_describe(big)
    W = 9 << 30
    for ws, n in ((None, 0), (None, need), (W, need - 1), (W + 128, need)):
        assert _status(run, big, P, Q, R, S, T, ws, n, None) == "LL_ERR_WORKSPACE"
    assert _status(run, big, P, Q, R, S, W, W, need, None) == "LL_ERR_INVALID_ARG"


# --- the binding ---------------------------------------------------------------

def test_the_binding_refuses():
    torch = pytest.importorskip("torch")
    ll = _ll()
    e4, f32 = torch.float8_e4m3fn, torch.float32
    x = torch.zeros(4, 16)
    for bad in (lambda: ll.rmsnorm(x, torch.ones(15)), lambda: ll.rmsnorm(x, torch.ones(16).half()),
                lambda: ll.rmsnorm(x, residual=torch.zeros(4, 15)), lambda: ll.rmsnorm(x, residual_out=x),
                lambda: ll.rmsnorm(x, residual=x.half()), lambda: ll.rmsnorm(x, out=x.half()),
                lambda: ll.rmsnorm(x.t()), lambda: ll.rmsnorm(x),  # not on a GPU
                lambda: ll.rmsnorm_grad(x, x, torch.zeros(3)), lambda: ll.rmsnorm_grad(x, x.half(), torch.zeros(4)),
                lambda: ll.rmsnorm_grad(x, x, torch.zeros(4), dh=x[:3]), lambda: ll.quant8(x), lambda: ll.quant8_pair(x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ll.rmsnorm8(x, dtype=f32), lambda: ll.quant8(x, dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    a, b = torch.zeros(4, 32).to(e4), torch.zeros(200, 32).to(e4)
    sa, sb, out = torch.ones(4, 1), torch.ones(2, 1), torch.zeros(4, 200)
    assert ll.gemm8_desc_for(a, sa, b, sb, out).b_block == 128
    assert ll.gemm8_desc_for(a, sa, b, torch.ones(200, 1), out).b_block == 1
    for args in ((a, sa, b, torch.ones(3, 1), out), (a, torch.ones(4, 2), b, sb, out), (a, sa[:3], b, sb, out),
                 (a, sa, b[:, :16], sb, out), (a, sa.double(), b, sb, out), (a, sa, b, sb, out[:3]),
                 (a, sa[:, 0], b, sb, out)):
        with pytest.raises(ValueError):
            ll.gemm8_desc_for(*args)
    with pytest.raises(TypeError):
        ll.gemm8_desc_for(a.float(), sa, b, sb, out)
