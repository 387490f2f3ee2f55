"""Root-mean-square norm, its 8-bit form and its gradients against the formulas in
64 bits.

Errors are counted in half steps u = 2^-24 of fp32.  A lane adds up at most 32
squares (rows of more than 16384: D / 1024 of them), then 6 lane exchanges and up
to 16 waves follow: the sum is off by (54 + D / 1024) u, rstd by half of that and 4
roundings more; h * rstd * gamma adds 2."""
import pytest

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 0), (1, 8192, 0), (3, 7, 1), (5, 128, 0), (2, 1000, 3), (70, 513, 8), (4, 5003, 3), (3, 8195, 0),
          (2, 16384, 8), (2, 16385, 0), (3, 40000, 5), (600, 64, 0)]


def _types():
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
            "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _rel(D):
    import helpers8 as h
    return ((54 + D / 1024) / 2 + 6) * h.U


def _formula(x, residual, gamma, eps):
    """(h as it is stored, y, rstd) in 64 bits."""
    import torch
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    v = h.double()
    rstd = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    g = 1.0 if gamma is None else gamma.double()
    return h, v * rstd * g, rstd[:, 0]


def _inputs(N, D, pad, dtype, residual, ptype, seed):
    import helpers8 as h
    x = h.normal((N, D), seed, dtype, 2.0)
    x[:, D // 3] *= 30.0
    r = h.normal((N, D), seed + 1, dtype, 1.0) if residual else None
    gamma = None if ptype is None else h.normal((D,), seed + 2, ptype, 0.3)
    dev = h.strided(x, pad)
    return x, r, gamma, dev, None if r is None else h.strided(r, pad), None if gamma is None else gamma.cuda()


def _close(got, want, rel, small=0.0):
    import torch
    got, want = got.cpu().double(), want.double()
    ok = (got - want).abs() <= want.abs() * rel + small
    assert bool(ok.all()), ((got - want).abs() - want.abs() * rel).max().item()
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("N,D,pad", SHAPES)
@pytest.mark.parametrize("type_", ["bf16", "f16", "f32"])
def test_norm(N, D, pad, type_):
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    t = _types()[type_]
    for residual, ptype in ((True, t), (False, torch.float32), (True, None)):
        x, r, gamma, dx, dr, dg = _inputs(N, D, pad, t, residual, ptype, N + D)
        want_h, want_y, want_r = _formula(x, r, gamma, 1e-6)
        y, got_h, rstd = ll.rmsnorm(dx, dg, residual=dr)
        if residual:
            assert torch.equal(got_h.cpu(), want_h)
        else:
            assert got_h is dx
        _close(rstd, want_r, _rel(D))
        _close(y, want_y, h.HALF_STEP[t] * (1 + 2 ** -10) + _rel(D), h.SMALL_STEP[t])


@pytest.mark.parametrize("N,D,pad", SHAPES)
@pytest.mark.parametrize("type_,q_type", [("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3")])
def test_norm8(N, D, pad, type_, q_type):
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    t, q8 = _types()[type_], _types()[q_type]
    for residual, ptype in ((True, t), (False, torch.float32)):
        x, r, gamma, dx, dr, dg = _inputs(N, D, pad, t, residual, ptype, N + D)
        want_h, want_y, want_r = _formula(x, r, gamma, 1e-6)
        q, scale, got_h, rstd = ll.rmsnorm8(dx, dg, residual=dr, dtype=q8)
        if residual:
            assert torch.equal(got_h.cpu(), want_h)
        _close(rstd, want_r, _rel(D))
        # scale = amax / F: the values' error and one rounding more
        _close(scale, h.block_amax(want_y, False) / h.LARGEST[q8], _rel(D) + h.U, 2.0 ** -126)
        small = h.expand(scale.cpu().double(), N, D, False) * h.SMALL_STEP[q8] * (1 + 2 ** -10)
        got = h.dequantise(q, scale, False)
        off = (got - want_y).abs() - small
        assert bool((off <= want_y.abs() * (h.HALF_STEP[q8] * (1 + 2 ** -10) + _rel(D) + 3 * h.U)).all())


def test_in_place_and_given_buffers():
    """residual_out over the residual or over x, out over x, and rows behind the last left alone."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    for D in (520, 20000):
        x, r = h.normal((5, D), 1, torch.bfloat16).cuda(), h.normal((5, D), 2, torch.bfloat16).cuda()
        g = h.normal((D,), 3, torch.bfloat16).cuda()
        y, s, rstd = ll.rmsnorm(x, g, residual=r)
        for into in ("r", "x"):
            x2, r2 = x.clone(), r.clone()
            y2, s2, rstd2 = ll.rmsnorm(x2, g, residual=r2, residual_out=r2 if into == "r" else x2)
            assert s2 is (r2 if into == "r" else x2)
            assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(rstd, rstd2)
            assert torch.equal(x2 if into == "r" else r2, x if into == "r" else r)
        want = ll.rmsnorm(x, g)[0]
        big = torch.full((7, D + 3), 9.0, dtype=torch.bfloat16, device="cuda")
        big[:5, :D] = x
        ll.rmsnorm(big[:5, :D], g, out=big[:5, :D])
        assert torch.equal(big[:5, :D], want) and bool((big[5:] == 9).all()) and bool((big[:, D:] == 9).all())


@pytest.mark.parametrize("D", [200, 8200, 17000])
def test_not_finite_stays_in_its_row(D):
    """A NaN or an infinity in a row, of x or of the residual, does not leave it."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    x, r = h.normal((6, D), 1, torch.bfloat16), h.normal((6, D), 2, torch.bfloat16)
    x[1, D // 2] = float("nan")
    r[3, D - 1] = float("inf")
    y, s, rstd = ll.rmsnorm(x.cuda(), residual=r.cuda())
    q, scale, _, _ = ll.rmsnorm8(x.cuda(), residual=r.cuda())
    good = [0, 2, 4, 5]
    for row in good:
        assert bool(torch.isfinite(y[row]).all()) and bool(torch.isfinite(scale[row]).all())
        assert bool(torch.isfinite(q[row].float()).all())
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(scale[1]).all())
    # infinity: rstd is 0, the row's finite values are 0 and the infinite one NaN
    assert bool(torch.isnan(y[3, D - 1])) and bool(torch.isnan(scale[3, -1])) and rstd[3].item() == 0


def test_rows_of_zeros():
    import torch
    import recsys_linear_layers_amd as ll
    x = torch.zeros(3, 300, dtype=torch.bfloat16, device="cuda")
    y, _, rstd = ll.rmsnorm(x)
    q, scale, _, _ = ll.rmsnorm8(x)
    assert bool((y == 0).all()) and bool((q.float() == 0).all()) and bool((scale == 2.0 ** -126).all())
    assert bool(((rstd - 1e3).abs() < 1e-2).all())


def _grad_formula(dy, hh, rstd, gamma, dh):
    """(dx, dgamma) and the sizes of the terms that were added up."""
    n = hh.double() * rstd.double()[:, None]
    g = dy.double() * (1.0 if gamma is None else gamma.double())
    m = (g * n).mean(1, keepdim=True)
    ma = (g * n).abs().mean(1, keepdim=True)
    dx = rstd.double()[:, None] * (g - n * m)
    size = rstd.double()[:, None] * (g.abs() + n.abs() * ma)
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    return dx, (dy.double() * n).sum(0), size, (dy.double() * n).abs().sum(0)


@pytest.mark.parametrize("N,D,pad", SHAPES)
@pytest.mark.parametrize("type_", ["bf16", "f16", "f32"])
def test_gradients(N, D, pad, type_):
    """dx: the terms' sizes times the errors of the row sum (as the squares' sum) and
    of six operations.  dgamma: N rows in some order, at most N roundings and 2 of
    each term."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    t = _types()[type_]
    for with_dh, ptype in ((True, t), (False, torch.float32), (True, None)):
        hh, dh, gamma, d_h, d_dh, d_g = _inputs(N, D, pad, t, with_dh, ptype, N + D)
        dy = h.normal((N, D), 5, t)
        rstd = (1.0 / torch.sqrt(hh.double().square().mean(1) + 1e-6)).float()
        dx, dgamma = ll.rmsnorm_grad(h.strided(dy, pad), d_h, rstd.cuda(), d_g, dh=d_dh)
        want, want_g, size, size_g = _grad_formula(dy, hh, rstd, gamma, dh)
        off = (dx.cpu().double() - want).abs()
        assert bool((off <= size * (2 * _rel(D) + 6 * h.U) + want.abs() * h.HALF_STEP[t] * (1 + 2 ** -10) + h.SMALL_STEP[t]).all())
        gt = gamma.dtype if gamma is not None else t
        off = (dgamma.cpu().double() - want_g).abs()
        assert dgamma.dtype == gt
        assert bool((off <= size_g * (N + 3) * h.U + want_g.abs() * h.HALF_STEP[gt] * (1 + 2 ** -10) + h.SMALL_STEP[gt]).all())
        alone, none = ll.rmsnorm_grad(h.strided(dy, pad), d_h, rstd.cuda(), d_g, dh=d_dh, param_grads=False)
        assert none is None and torch.equal(alone, dx)


def test_gradients_against_differences():
    """Central differences of sum(c y) + sum(e h) in 64 bits; step 1e-4 of values of
    size 1: 1e-8 of curvature beside fp32's rounding."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    N, D, eps = 3, 9, 1e-3
    x, r, g = h.normal((N, D), 1).double(), h.normal((N, D), 2).double(), h.normal((D,), 3).double()
    x, r, g = x.float().double(), r.float().double(), g.float().double()
    c, e = h.normal((N, D), 4), h.normal((N, D), 5)

    def loss(x, r, g):
        s = x + r
        return ((c.double() * s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * g).sum() + (e.double() * s).sum()).item()

    _, hh, rstd = ll.rmsnorm(x.float().cuda(), g.float().cuda(), residual=r.float().cuda(), eps=eps)
    dx, dgamma = ll.rmsnorm_grad(c.cuda(), hh, rstd, g.float().cuda(), dh=e.cuda())
    for grad, which, n in ((dx, 0, (N, D)), (dx, 1, (N, D)), (dgamma, 2, (D,))):
        for i in range(grad.numel()):
            args = [x.clone(), r.clone(), g.clone()]
            args[which].view(-1)[i] += 1e-4
            up = loss(*args)
            args[which].view(-1)[i] -= 2e-4
            assert abs((up - loss(*args)) / 2e-4 - grad.reshape(-1)[i].item()) < 1e-5, (which, i)


def test_gradient_in_place_and_empty():
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    for D in (300, 20000):
        dy, hh, dh = (h.normal((4, D), k, torch.bfloat16).cuda() for k in (1, 2, 3))
        rstd = torch.rand(4, device="cuda") + 0.5
        want, _ = ll.rmsnorm_grad(dy, hh, rstd, dh=dh)
        into = dh.clone()
        got, _ = ll.rmsnorm_grad(dy, hh, rstd, dh=into, out=into)
        assert got is into and torch.equal(got, want)
    e = torch.empty(0, 40, device="cuda")
    dx, dgamma = ll.rmsnorm_grad(e, e, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 40) and bool((dgamma == 0).all())
    y, hh, rstd = ll.rmsnorm(e)
    assert y.shape == (0, 40) and rstd.shape == (0,)
    y, hh, rstd = ll.rmsnorm(torch.empty(4, 0, device="cuda"))
    assert y.shape == (4, 0)


def test_equal_bits_whatever_the_workspace_held():
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    dy, hh = h.normal((1500, 1100), 1, torch.bfloat16).cuda(), h.normal((1500, 1100), 2, torch.bfloat16).cuda()
    rstd = torch.rand(1500, device="cuda") + 0.5
    dx, dg = torch.empty_like(hh), torch.empty(1100, dtype=torch.bfloat16, device="cuda")
    desc = ll.RmsnormGradDesc(1500, 1100, 1100, 1100, 0, 1100, ll.LL_BF16, ll.LL_BF16)
    need = ll.rmsnorm_grad_workspace_size(desc)
    first = None
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        ll.rmsnorm_grad_run(desc, dy.data_ptr(), hh.data_ptr(), None, rstd.data_ptr(), None, dx.data_ptr(),
                            dg.data_ptr(), ws.data_ptr(), need)
        got = (dx.clone(), dg.clone())
        first = first or got
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])
