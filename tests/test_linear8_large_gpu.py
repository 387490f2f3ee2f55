"""The 8-bit linear layers' operators where a workgroup takes several rows or tiles,
and where offsets pass 32 bits."""
import pytest

pytestmark = pytest.mark.gpu

# rows per workgroup and step: 4 (D up to 2048), 1 (beyond); more rows than any launch has workgroups
MANY = [(9001, 300, 3), (12001, 2040, 0), (5003, 2100, 1), (4099, 5003, 3), (3001, 8200, 8), (1500, 16384, 0),
        (17000, 17000, 0)]


def _tests():
    import test_rmsnorm_gpu
    return test_rmsnorm_gpu


def _normal(shape, seed, dtype, std=1.0, pad=0):
    """On the GPU, in rows of pad more elements."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, d = shape
    t = torch.empty((n, d + pad), dtype=dtype, device="cuda")[:, :d]
    for r in range(0, n, 4096):
        t[r:r + 4096] = (torch.randn((min(4096, n - r), d), generator=g, device="cuda") * std).to(dtype)
    return t


def _norm_rows(x, r, gamma, rows):
    """The formula of some rows, in 64 bits."""
    import torch
    h = x[rows] if r is None else (x[rows].double() + r[rows].double()).to(x.dtype)
    v = h.double()
    rstd = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    return h, v * rstd * gamma.double(), rstd[:, 0]


@pytest.mark.parametrize("N,D,pad", MANY)
@pytest.mark.parametrize("type_", ["bf16", "f32"])
def test_norm_of_many_rows(N, D, pad, type_):
    """Every row's sums are its own; tolerances as for few rows."""
    import torch
    import helpers8 as h
    import recsys_linear_layers_amd as ll
    T = _tests()
    t = T._types()[type_]
    x, r = _normal((N, D), 1, t, 2.0, pad), _normal((N, D), 2, t, 1.0, pad)
    gamma = _normal((1, D), 3, t)[0].contiguous()
    y, s, rstd = ll.rmsnorm(x, gamma, residual=r)
    q, scale, s8, rstd8 = ll.rmsnorm8(x, gamma, residual=r)
    assert torch.equal(s, s8) and torch.equal(rstd, rstd8)
    for a in range(0, N, 2048):
        rows = slice(a, a + 2048)
        want_h, want_y, want_r = _norm_rows(x, r, gamma, rows)
        assert torch.equal(s[rows], want_h)
        assert bool(((rstd[rows].double() - want_r).abs() <= want_r * T._rel(D)).all())
        off = (y[rows].double() - want_y).abs() - want_y.abs() * (h.HALF_STEP[t] * (1 + 2 ** -10) + T._rel(D))
        assert bool((off <= h.SMALL_STEP[t]).all())
        e4 = torch.float8_e4m3fn
        each = scale[rows].double().repeat_interleave(128, 1)[:, :D]
        off = (q[rows].double() * each - want_y).abs() - want_y.abs() * (h.HALF_STEP[e4] * (1 + 2 ** -10) + T._rel(D) + 3 * h.U)
        assert bool((off <= each * h.SMALL_STEP[e4] * (1 + 2 ** -10)).all())
    for into in (r, x):  # h over either, then y over x: rows are read ahead of the writes
        x2, r2 = x.clone(), r.clone()
        y2, s2, _ = ll.rmsnorm(x2, gamma, residual=r2, residual_out=r2 if into is r else x2)
        assert torch.equal(y2, y) and torch.equal(s2, s)
    alone = ll.rmsnorm(x, gamma)[0]
    x2 = x.clone()
    assert torch.equal(ll.rmsnorm(x2, gamma, out=x2)[0], alone)


@pytest.mark.parametrize("N,D,pad", MANY)
@pytest.mark.parametrize("type_", ["bf16", "f32"])
def test_gradients_of_many_rows(N, D, pad, type_):
    import torch
    import helpers8 as h
    import recsys_linear_layers_amd as ll
    T = _tests()
    t = T._types()[type_]
    hh, dy, dh = _normal((N, D), 1, t, 2.0, pad), _normal((N, D), 2, t, 1.0, pad), _normal((N, D), 3, t, 1.0, pad)
    gamma = _normal((1, D), 4, t)[0].contiguous()
    rstd = torch.cat([(1.0 / torch.sqrt(hh[a:a + 2048].double().square().mean(1) + 1e-6)).float() for a in range(0, N, 2048)])
    dx, dgamma = ll.rmsnorm_grad(dy, hh, rstd, gamma, dh=dh)
    want_g = size_g = 0
    for a in range(0, N, 2048):
        rows = slice(a, a + 2048)
        want, part, size, part_size = T._grad_formula(dy[rows], hh[rows], rstd[rows], gamma, dh[rows])
        want_g, size_g = want_g + part, size_g + part_size
        off = (dx[rows].double() - want).abs()
        assert bool((off <= size * (2 * T._rel(D) + 6 * h.U) + want.abs() * h.HALF_STEP[t] * (1 + 2 ** -10) + h.SMALL_STEP[t]).all())
    off = (dgamma.double() - want_g).abs()
    assert bool((off <= size_g * (N + 3) * h.U + want_g.abs() * h.HALF_STEP[t] * (1 + 2 ** -10) + h.SMALL_STEP[t]).all())
    into = dh.clone()
    again, dgamma2 = ll.rmsnorm_grad(dy, hh, rstd, gamma, dh=into, out=into)
    assert torch.equal(again, dx) and torch.equal(dgamma2, dgamma)


def _far(t, ld):
    """The same values in rows ld elements apart (what lies between is not set)."""
    import torch
    n, d = t.shape
    buf = torch.empty(n * ld, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
    out = (buf.view(t.dtype) if t.element_size() == 1 else buf).view(n, ld)[:, :d]
    out.copy_(t)
    return out


def test_rows_far_apart():
    """Row starts beyond 2^32 elements: the same bits as from rows side by side."""
    import torch
    import recsys_linear_layers_amd as ll
    n, d, ld = 1100, 300, 1 << 22
    x, r, dy = (_normal((n, d), k, torch.bfloat16) for k in (1, 2, 3))
    gamma = _normal((1, d), 4, torch.bfloat16)[0].contiguous()
    y, s, rstd = ll.rmsnorm(x, gamma, residual=r)
    fx, fr = _far(x, ld), _far(r, ld)
    into, out = _far(torch.zeros_like(x), ld), _far(torch.zeros_like(x), ld)
    y2, s2, rstd2 = ll.rmsnorm(fx, gamma, residual=fr, residual_out=into, out=out)
    assert y2 is out and s2 is into
    assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(rstd2, rstd)
    dx, dg = ll.rmsnorm_grad(dy, s, rstd, gamma, dh=r)
    dx2, dg2 = ll.rmsnorm_grad(_far(dy, ld), into, rstd, gamma, dh=fr, out=out)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg)
    for squares in (False, True):
        for a, b in zip(ll.quant8_pair(x, squares=squares), ll.quant8_pair(fx, squares=squares)):
            assert torch.equal(a.reshape(-1).view(torch.uint8) if a.element_size() == 1 else a,
                               b.reshape(-1).view(torch.uint8) if b.element_size() == 1 else b)


@pytest.mark.parametrize("M,N", [(5, 1100), (60, 1100), (1100, 1040)])
def test_product_of_rows_far_apart(M, N):
    import torch
    import recsys_linear_layers_amd as ll
    K, ld = 300, (1 << 22) - 16
    a, sa = ll.quant8(_normal((M, K), 1, torch.float32))
    b, sb = ll.quant8(_normal((N, K), 2, torch.float32), squares=True)
    fa, fb = _far(a, ld), _far(b, ld)
    for c in (torch.bfloat16, torch.float32):
        want = ll.gemm8(a, sa, b, sb, out_dtype=c)
        out = torch.empty((M, 1 << 22), dtype=c, device="cuda")[:, :N]
        assert torch.equal(ll.gemm8(fa, sa, fb, sb, out=out), want)


def test_more_tiles_than_a_launch_has():
    """A column of 2^29 values: 2^22 tiles of 128 rows and a few more."""
    import torch
    import recsys_linear_layers_amd as ll
    n = ((1 << 22) + 3) * 128 + 5
    x = torch.zeros((n, 1), dtype=torch.bfloat16, device="cuda")
    tail = 128 * 1000
    start = n // 128 * 128 - tail
    x[start:] = _normal((n - start, 1), 1, torch.bfloat16)
    x[:tail] = _normal((tail, 1), 2, torch.bfloat16)
    q, s, qt, st = ll.quant8_pair(x)
    for part in (slice(0, tail), slice(start, n)):
        q1, s1, qt1, st1 = ll.quant8_pair(x[part])
        assert torch.equal(q[part].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[part], s1)
        assert torch.equal(qt[:, part].view(torch.uint8), qt1.view(torch.uint8))
        assert torch.equal(st[:, part.start // 128:-(-part.stop // 128)], st1)
    assert bool((st[:, 1000:start // 128] == 2.0 ** -126).all())


def test_nan_stays_in_its_tile(monkeypatch):
    """A workgroup that goes on from a tile with NaN to another."""
    import torch
    import recsys_linear_layers_amd as ll
    K = 300
    for kind, bm, bn in (("TILE64x128", 64, 128), ("TILE128x128", 128, 128), ("TILE256x256", 256, 256)):
        monkeypatch.setenv("LL_GEMM8_KIND", kind)
        M, N = 9 * bm - 5, 61 * bn - 3
        a, sa = ll.quant8(_normal((M, K), 1, torch.float32))
        for squares in (True, False):
            b, sb = ll.quant8(_normal((N, K), 2, torch.float32), squares=squares)
            for c in (torch.bfloat16, torch.float32):
                clean = ll.gemm8(a, sa, b, sb, out_dtype=c)
                bad = sa.clone()
                bad[M // 2, 2] = float("nan")
                got = ll.gemm8(a, bad, b, sb, out_dtype=c)
                assert bool(torch.isnan(got[M // 2]).all())
                got[M // 2] = clean[M // 2]
                assert torch.equal(got, clean)
