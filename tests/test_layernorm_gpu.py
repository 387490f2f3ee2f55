"""Layer norm and its gradients against their definitions in 64 bits.

Tolerances, with u = 2^-24 and h = eps(type) / 2.  A sum over the D columns of
a row passes through at most k = D/64 + 30 roundings per term (a lane's own
columns one after the other, then trees over lanes and waves; wider rows use
more lanes), so a mean is off by at most k u times the mean magnitude, and the
variance around it, whose error from the mean's is of second order, by (k + 3)
u of itself.  Each elementwise step adds one u of its operands, the store h of
the result.  Factors of two stand for the second-order terms."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = ["bfloat16", "float16", "float32"]


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


def _half(dt):
    import torch
    return torch.finfo(dt).eps / 2


def _tiny(dt):
    import torch
    return 2.0 ** -25 if dt == torch.float16 else 0.0


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _within(got, ref, tol, what):
    import torch
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), what
    worst = (err / tol.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert bool((err <= tol).all()), f"{what}: err/tol {worst:.3g}"


def _strided(rows, cols, pad, dt, g, offset=0.0):
    import torch
    t = torch.randn((rows, cols + pad), generator=g, device="cuda", dtype=torch.float32) + offset
    return t.to(dt)[:, :cols]


def _params(D, kind, dt, g):
    import torch
    if kind == "none":
        return None, None
    pt = torch.float32 if kind == "f32" else dt
    return ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt),
            (0.3 * torch.randn(D, generator=g, device="cuda")).to(pt))


def _forward_check(x, gamma, beta, eps, out, what):
    import torch
    y, mean, rstd = out
    N, D = x.shape
    e = torch.tensor(eps, dtype=torch.float32).double().item()
    xd = x.double()
    m = xd.mean(1)
    v = ((xd - m[:, None]) ** 2).mean(1)
    r = (v + e) ** -0.5
    k = D / 64 + 30
    me = k * U * xd.abs().mean(1) + U * m.abs()
    _within(mean, m, me * 1.01, what + " mean")
    re = r * (U * (k / 2 + 6) + (me * r) ** 2)
    _within(rstd, r, re * 1.01, what + " rstd")
    ga = gamma.double() if gamma is not None else torch.ones(D, dtype=torch.float64, device="cuda")
    be = beta.double() if beta is not None else torch.zeros(D, dtype=torch.float64, device="cuda")
    xhat = (xd - m[:, None]) * r[:, None]
    ref = xhat * ga + be
    tol = (ref.abs() * (_half(x.dtype) + 2 * U)
           + 2 * ga.abs() * (xhat.abs() * (re / r + 3 * U)[:, None] + (me * r)[:, None])) * 1.01 + _tiny(x.dtype)
    _within(y, ref, tol, what + " y")


def _grad_check(dy, x, gamma, mean, rstd, got, what):
    import torch
    dx, dgamma, dbeta = got
    N, D = x.shape
    dt = x.dtype
    ga = gamma.double() if gamma is not None else torch.ones(D, dtype=torch.float64, device="cuda")
    r = rstd.double()[:, None]
    n = (x.double() - mean.double()[:, None]) * r
    h = dy.double() * ga
    m1, m2 = h.mean(1, keepdim=True), (h * n).mean(1, keepdim=True)
    ref = r * (h - m1 - n * m2)
    k = D / 64 + 34
    a1, a2 = h.abs().mean(1, keepdim=True), (h * n).abs().mean(1, keepdim=True)
    inner = 4 * (h.abs() + m1.abs() + (n * m2).abs()) + k * (a1 + n.abs() * a2) + 4 * n.abs() * a2
    _within(dx, ref, ref.abs() * (_half(dt) + U) + 1.01 * U * r * inner + _tiny(dt), what + " dx")
    if dgamma is None:
        return
    pt = dgamma.dtype
    depth = min(N, N / 256 + 160) + 8
    ref, S = (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)
    _within(dgamma, ref, ref.abs() * _half(pt) + 1.01 * depth * U * S + _tiny(pt), what + " dgamma")
    ref, S = dy.double().sum(0), dy.double().abs().sum(0)
    _within(dbeta, ref, ref.abs() * _half(pt) + 1.01 * depth * U * S + _tiny(pt), what + " dbeta")


# one column, a lane's, a wave's and a workgroup's widths and one beyond each;
# 16384 columns are the widest row held in registers
SIZES = [(1, 1, 0), (3, 2, 0), (5, 64, 0), (2, 65, 1), (9, 512, 0), (4, 520, 8), (7, 1001, 0), (130, 1024, 0),
         (3, 2048, 0), (3, 2056, 0), (5, 4096, 0), (2, 4099, 5), (6, 5003, 0), (3, 8192, 0), (2, 8200, 0),
         (3, 16384, 0), (2, 16383, 0), (2, 16392, 8), (1, 33333, 0), (1500, 72, 0)]


@pytest.mark.parametrize("params", ["same", "f32", "none"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,D,pad", SIZES)
def test_forward_and_gradients(N, D, pad, dtype, params):
    import torch
    ll = _ll()
    dt, g = getattr(torch, dtype), _gen(N * 31 + D)
    x = _strided(N, D, pad, dt, g, offset=0.5)
    gamma, beta = _params(D, params, dt, g)
    what = f"{dtype} {N}x{D}+{pad} {params}"
    out = ll.layernorm(x, gamma, beta, eps=1e-5)
    _forward_check(x, gamma, beta, 1e-5, out, what)
    dy = _strided(N, D, pad, dt, g)
    got = ll.layernorm_grad(dy, x, out[1], out[2], gamma)
    _grad_check(dy, x, gamma, out[1], out[2], got, what)
    again = ll.layernorm_grad(dy, x, out[1], out[2], gamma)
    for p, q in zip(got, again):
        assert torch.equal(p, q), what + ": equal inputs, other bits"


@pytest.mark.parametrize("dtype", TYPES)
def test_more_rows_than_workgroups(dtype):
    import torch
    ll = _ll()
    dt, g = getattr(torch, dtype), _gen(3)
    for N, D in ((3000, 300), (1100, 2304), (5001, 65), (700, 17000)):
        x, dy = _strided(N, D, 0, dt, g), _strided(N, D, 0, dt, g)
        gamma, beta = _params(D, "f32", dt, g)
        out = ll.layernorm(x, gamma, beta)
        _forward_check(x, gamma, beta, 1e-5, out, f"{dtype} {N}x{D}")
        _grad_check(dy, x, gamma, out[1], out[2], ll.layernorm_grad(dy, x, out[1], out[2], gamma), f"{dtype} {N}x{D}")


def test_rows_of_equal_values_and_far_from_zero():
    """A constant row has variance 0: y = beta.  A row far from zero keeps the
    precision of the differences (variance around the mean, not E[x^2] - mean^2)."""
    import torch
    ll = _ll()
    D = 1000
    beta = torch.linspace(-1, 1, D, device="cuda")
    x = torch.full((2, D), 3.0, device="cuda")
    y, mean, rstd = ll.layernorm(x, None, beta, eps=1e-5)
    assert torch.equal(y, beta.expand(2, D)) and torch.equal(mean, torch.full((2,), 3.0, device="cuda"))
    g = _gen(8)
    x = 4096.0 + torch.randint(-8, 9, (4, D), generator=g, device="cuda").float()
    _forward_check(x, None, None, 1e-5, ll.layernorm(x), "far from zero")


def test_in_place_and_dx_alone():
    import torch
    ll = _ll()
    g = _gen(4)
    for D in (96, 5000, 20000):
        x = _strided(7, D, 0, torch.bfloat16, g)
        want, mean, rstd = ll.layernorm(x)
        dy = _strided(7, D, 0, torch.bfloat16, g)
        full = ll.layernorm_grad(dy, x, mean, rstd)
        part = ll.layernorm_grad(dy, x, mean, rstd, param_grads=False)
        assert part[1] is None and part[2] is None and torch.equal(part[0], full[0])
        y = x.clone()
        assert torch.equal(ll.layernorm(y, out=y)[0], want)


def test_no_rows():
    import torch
    ll = _ll()
    for D in (48, 20000):
        x = torch.empty((0, D), device="cuda")
        y, mean, rstd = ll.layernorm(x)
        assert y.shape == (0, D) and mean.shape == (0,)
        dx, dg, db = ll.layernorm_grad(x, x, mean, rstd)
        assert dx.shape == (0, D) and float(dg.abs().max()) == 0 and float(db.abs().max()) == 0


def test_nan_stays_in_its_row():
    import torch
    ll = _ll()
    g = _gen(6)
    for D in (100, 3000):
        x = _strided(9, D, 0, torch.float32, g)
        want = ll.layernorm(x)[0]
        bad = x.clone()
        bad[4, 7] = float("nan")
        bad[5, 3] = float("inf")
        y = ll.layernorm(bad)[0]
        keep = [0, 1, 2, 3, 6, 7, 8]
        assert torch.equal(y[keep], want[keep]) and bool(y[4].isnan().all())


def test_gradients_agree_with_differences():
    """sum(y * R) by central differences in 64 bits of the definition."""
    import torch
    ll = _ll()
    g = _gen(12)
    N, D, eps, step = 3, 10, 1e-5, 1e-4
    x = torch.randn((N, D), generator=g, device="cuda")
    gamma, beta = _params(D, "f32", torch.float32, g)
    R = torch.randn((N, D), generator=g, device="cuda")

    def f(x, ga, be):
        m = x.mean(1, keepdim=True)
        v = ((x - m) ** 2).mean(1, keepdim=True)
        return float((((x - m) * (v + eps) ** -0.5 * ga + be) * R.double()).sum())

    _, mean, rstd = ll.layernorm(x, gamma, beta, eps=eps)
    got = ll.layernorm_grad(R, x, mean, rstd, gamma)
    args = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate(got):
        for j in range(args[i].numel()):
            plus, minus = [a.clone() for a in args], [a.clone() for a in args]
            plus[i].view(-1)[j] += step
            minus[i].view(-1)[j] -= step
            num = (f(*plus) - f(*minus)) / (2 * step)
            # central differences are off by step^2 times a third derivative of order 10 here
            assert abs(num - float(grad.reshape(-1)[j])) <= 1e-5 * (1 + abs(num))


def test_streams_and_graph():
    import torch
    ll = _ll()
    g = _gen(15)
    for D in (1024, 6000):
        x, dy = _strided(600, D, 0, torch.bfloat16, g), _strided(600, D, 0, torch.bfloat16, g)
        gamma, beta = _params(D, "f32", torch.bfloat16, g)
        y, mean, rstd = ll.layernorm(x, gamma, beta)
        want = ll.layernorm_grad(dy, x, mean, rstd, gamma)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = ll.layernorm_grad(dy, x, mean, rstd, gamma)
        torch.cuda.current_stream().wait_stream(side)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y2, mean2, rstd2 = ll.layernorm(x, gamma, beta)
            got = ll.layernorm_grad(dy, x, mean2, rstd2, gamma)
        for _ in range(3):
            for t in (y2, mean2, rstd2, *got):
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y2, y)
            for p, q in zip(got, want):
                assert torch.equal(p, q)
            torch.randn(64, 64, device="cuda").sum().item()


def test_more_than_2_to_31_elements():
    import torch
    ll = _ll()
    N, D = 2 ** 18 + 5, 8192
    x = torch.zeros((N, D), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, D), device="cuda").to(torch.bfloat16)
    y, mean, rstd = ll.layernorm(x)
    _forward_check(x[-3:], None, None, 1e-5, (y[-3:], mean[-3:], rstd[-3:]), "last rows")
    assert float(y[: 10].abs().max()) == 0
