"""The vocabulary cross entropy and its gradients against their definitions in
64 bits.

Tolerances, with u = 2^-24, h = eps(type) / 2 of the operands' 16-bit type and
q of an output's type.  A logit is a sum of D exact products added in fp32: off
by at most (D + 2) u A, A = sum |x w| (the target's likewise).  The log of the
sum of V exponentials carries the largest of the logits' errors, the rounding
of its argument differences and of the sum (V terms; 2 log2 V + 40 roundings
each, in trees), and its own.  The exponentials are the hardware's: 2^-22
relative plus the rounding of an argument r, |r| 2 u.  dz is then off by that
error of z - lse relative to p, once h of itself for its rounding, and once
2^-11 of p where its numerator was kept in fp16 (down to 2^-29 of the largest
numerator of its part, which is at most 1; below, 2^-40 absolute); with fp16
it is scaled first, so that only values below 2^-14 / 2^13 of the largest
|dloss| lose bits: at most 2^-25 / 2^13 of it.  The products add (V + 2) u or
(N + 2) u of the sum of magnitudes, and q of the result.  What is smaller than
a normal fp32 or bf16 number, 2^-126, may be lost (the exponential, dz, an
output)."""
import math

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


def _half(dt):
    import torch
    return torch.finfo(dt).eps / 2


def _tiny(dt):
    import torch
    return 2.0 ** -25 if dt == torch.float16 else 2.0 ** -126


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


def _strided(rows, cols, pad, dt, g, std=1.0):
    import torch
    return (torch.randn((rows, cols + pad), generator=g, device="cuda") * std).to(dt)[:, :cols]


def _check(x, w, target, dloss, out, ignore, what):
    """out: (loss, lse, dx, dw), the gradients perhaps None."""
    import torch
    loss, lse, dx, dw = out
    (N, D), V = x.shape, w.shape[0]
    live = (target >= 0) & (target < V) & (target != ignore)
    assert float(loss[~live].abs().sum()) == 0 and float(lse[~live].abs().sum()) == 0
    if dx is not None:
        assert float(dx[~live].float().abs().sum()) == 0
    xd, wd = x[live].double(), w.double()
    t = target[live]
    z = xd @ wd.T
    A = xd.abs() @ wd.abs().T
    ez = (D + 2) * U * A
    ref = torch.logsumexp(z, 1)
    spread = (z - ref[:, None])
    p = torch.exp(spread)
    elog = ez + 2 * U * spread.abs() + 2.0 ** -22
    tol = (p * elog).sum(1) + (2 * math.log2(V) + 40) * U + 4 * U * ref.abs()
    _within(lse[live], ref, 1.01 * tol, what + " lse")
    at = t[:, None]
    zt, et = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
    _within(loss[live], ref - zt, 1.01 * (tol + et + 2 * U * (ref.abs() + zt.abs())), what + " loss")
    if dx is None and dw is None:
        return
    h = _half(x.dtype)
    g = dloss[live].double()[:, None]
    dz = p.clone()
    dz.scatter_add_(1, at, -torch.ones_like(zt)[:, None])
    dz *= g
    kept = p * 2.0 ** -11 + 2.0 ** -40
    ed = ((p * (elog + tol[:, None] + 2 * U * spread.abs() + 4 * U) + kept) * g.abs() + dz.abs() * (h + 4 * U)) * 1.01
    ed += 2.0 ** -126 * (1 + g.abs())
    if x.dtype == torch.float16:
        ed += 2.0 ** -38 * float(dloss.abs().max())
    if dx is not None:
        r = dz @ wd
        tol = ed @ wd.abs() + (V + 2) * U * ((dz.abs() + ed) @ wd.abs()) + r.abs() * _half(dx.dtype) + _tiny(dx.dtype)
        _within(dx[live], r, 1.01 * tol, what + " dx")
    if dw is not None:
        r = dz.T @ xd
        tol = ed.T @ xd.abs() + (N + 2) * U * ((dz.abs() + ed).T @ xd.abs()) + r.abs() * _half(dw.dtype) + _tiny(dw.dtype)
        _within(dw, r, 1.01 * tol, what + " dw")


def _case(N, V, D, dtype, pad=0, seed=0, std=1.5, ignored=0.2):
    import torch
    dt, g = getattr(torch, dtype), _gen(seed + N + V + D)
    x = _strided(N, D, pad, dt, g)
    w = _strided(V, D, pad, dt, g, std / math.sqrt(D))
    target = torch.randint(0, V, (N,), generator=g, device="cuda")
    target[torch.rand(N, generator=g, device="cuda") < ignored] = -100
    dloss = torch.rand(N, generator=g, device="cuda") * 2 - 0.5
    return x, w, target, dloss


# one row; widths off whole 8s and 64s; vocabularies below, at and beyond whole
# tiles; enough rows and tiles for the large-tile products
SIZES = [(1, 1, 8, 0), (1, 1000, 64, 0), (2, 300, 1, 0), (5, 257, 72, 8), (16, 4096, 128, 0), (65, 777, 100, 0),
         (130, 2001, 1000, 3), (300, 50, 33, 0), (257, 5003, 192, 0), (700, 1025, 96, 0), (1, 40000, 520, 0),
         (1030, 4100, 320, 0), (2048, 8192, 64, 0), (4, 3, 5000, 0), (4100, 2050, 72, 0), (300, 20000, 128, 8),
         (1200, 9999, 200, 0), (513, 12801, 1088, 0), (2048, 8192, 192, 0), (4100, 2050, 136, 0), (70, 900, 150, 0)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("N,V,D,pad", SIZES)
def test_loss_and_gradients(N, V, D, pad, dtype):
    import torch
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, pad)
    what = f"{dtype} {N}x{V}x{D}+{pad}"
    loss, lse = ll.vocab_xent(x, w, target)
    _check(x, w, target, None, (loss, lse, None, None), -100, what)
    out = ll.vocab_xent_grad(x, w, target, dloss)
    _check(x, w, target, dloss, out, -100, what)
    for a, b in zip(ll.vocab_xent_grad(x, w, target, dloss), out):
        assert torch.equal(a, b), what + ": equal inputs, other bits"


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("N,V,D,pad", [(1, 15, 3, 0), (3, 17, 40, 0), (7, 1000, 33, 5), (16, 1001, 4096, 0),
                                       (16, 70000, 264, 8), (2, 4099, 8192, 0), (17, 4099, 256, 0), (9, 300, 8200, 0),
                                       (32, 5000, 1001, 3), (33, 40000, 520, 0), (64, 2000, 64, 0), (65, 33000, 129, 0),
                                       (128, 1111, 512, 0), (128, 3000, 640, 0), (129, 900, 64, 0)])
def test_few_rows(N, V, D, pad, dtype):
    """Up to 64 rows (as far as x fits) stream the vocabulary once; 65 do not."""
    import torch
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, pad, ignored=0.1)
    few = N <= 64 and N * (-(-D // 32) * 32 + 8) * 2 <= 144 * 1024
    assert ("few_rows" in ll.xent_plan_for(x, w).describe()) == few
    what = f"{dtype} {N}x{V}x{D}+{pad}"
    loss, lse = ll.vocab_xent(x, w, target)
    _check(x, w, target, None, (loss, lse, None, None), -100, what)
    _check(x, w, target, dloss, ll.vocab_xent_grad(x, w, target, dloss), -100, what)
    bad, t = x.clone(), target.clone()
    bad[-1], t[-1] = float("nan"), V
    got = ll.vocab_xent(bad, w, t)
    assert torch.equal(got[0][:-1], loss[:-1]) and float(got[0][-1]) == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("N,V,D,pad", [(65, 1, 1, 0), (65, 63, 7, 0), (66, 65, 8, 0), (127, 2001, 9, 1), (128, 5000, 63, 0),
                                       (129, 64, 65, 0), (300, 20001, 64, 3), (1000, 127, 127, 0), (777, 3001, 128, 8),
                                       (5000, 129, 33, 0), (70, 60000, 100, 0), (40000, 300, 40, 0), (200, 70000, 16, 0)])
def test_narrow_rows(N, V, D, pad, dtype):
    """More than 64 rows of up to 128 columns: no logits are stored, whatever the bound on a piece."""
    import torch
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, pad, ignored=0.1)
    plan = ll.xent_plan_for(x, w, x.clone(), w.clone())
    assert plan.describe().startswith("narrow")
    what = f"{dtype} {N}x{V}x{D}+{pad}"
    loss, lse = ll.vocab_xent(x, w, target)
    _check(x, w, target, None, (loss, lse, None, None), -100, what)
    out = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=1)
    _check(x, w, target, dloss, out, -100, what)
    f = ll.vocab_xent_grad(x, w, target, dloss, dx=torch.empty((N, D + 3), device="cuda")[:, :D],
                           dw=torch.empty((V, D), device="cuda"))
    _check(x, w, target, dloss, f, -100, what + " fp32")
    assert torch.equal(out[0], loss) and torch.equal(f[0], loss)
    # what rows without a target hold stays out of dw, a NaN in its row's loss
    bad = torch.where((target == -100)[:, None], float("nan"), x)
    got = ll.vocab_xent_grad(bad, w, target, dloss)
    assert torch.equal(got[3], out[3]) and torch.equal(got[0], loss)
    # a whole vocabulary of -inf but for two entries
    w2 = torch.full_like(w, float("-inf"))
    w2[0] = w2[V // 2] = 0
    ones = torch.ones_like(x)
    t = torch.where(target >= 0, torch.where(target % 2 == 0, 0, V // 2), target)
    loss, lse = ll.vocab_xent(ones, w2, t)
    want = torch.where(t >= 0, math.log(2.0 if V > 1 else 1.0), 0.0).float()
    assert torch.allclose(loss, want, rtol=1e-6) and torch.equal(loss, lse)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("V,D", [(1, 8), (1000, 64), (40000, 520), (5001, 333)])
def test_one_row_with_a_target(V, D, dtype):
    ll = _ll()
    x, w, target, dloss = _case(1, V, D, dtype, ignored=0.0)
    _check(x, w, target, dloss, ll.vocab_xent_grad(x, w, target, dloss), -100, f"one row {V}x{D}")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("N,V,D,pieces", [(40, 1111, 64, 5), (300, 3000, 136, 3), (1, 700, 40, 3), (1024, 9000, 136, 4)])
def test_pieces_of_the_vocabulary(N, V, D, pieces, dtype):
    """A bound that holds a fraction of the vocabulary: the pieces join to the same."""
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, seed=5)
    plan = ll.xent_plan_for(x, w, x.clone(), w.clone(), piece_bytes=1)
    assert "pieces=%d " % (-(-V // 256)) in plan.describe(), plan.describe()
    out = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=1)
    _check(x, w, target, dloss, out, -100, f"256 columns {dtype}")
    bound = N * 6 * (-(-V // pieces // 256) * 256)
    out = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
    _check(x, w, target, dloss, out, -100, f"{pieces} pieces {dtype}")
    loss, lse = ll.vocab_xent(x, w, target, piece_bytes=1)
    _check(x, w, target, None, (loss, lse, None, None), -100, f"256 columns {dtype}")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_numerators_kept_for_some_pieces(dtype):
    """Large enough for the softmax in the product: some pieces keep their
    numerators, the logits of the others are formed again; the last is short."""
    ll = _ll()
    N, V, D = 2000, 9000, 192
    x, w, target, dloss = _case(N, V, D, dtype, seed=6)
    for cols, pieces, kept in ((1024, 9, 4), (1280, 8, 4), (256, 36, 4), (2048, 5, 4)):
        # a column takes 2 bytes per padded row, and with fp16 4 per column of the dw that is scaled afterwards
        bound = 4 * cols * (2 * 2048 + (4 * D if dtype == "float16" else 0))
        plan = ll.xent_plan_for(x, w, x.clone(), w.clone(), piece_bytes=bound).describe()
        assert "fused=1" in plan and f"pieces={pieces} " in plan, plan
        assert f"kept={kept} " in plan or dtype == "float16", plan
        out = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
        _check(x, w, target, dloss, out, -100, f"{dtype} pieces of {cols}")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_one_gradient_alone_and_fp32_gradients(dtype):
    import torch
    ll = _ll()
    for N, V, D, bound in ((70, 600, 96, 0), (70, 600, 96, 1), (600, 2100, 128, 0), (600, 2100, 128, 1),
                           (600, 2100, 192, 0), (600, 2100, 192, 1)):
        x, w, target, dloss = _case(N, V, D, dtype, seed=9)
        both = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
        a = ll.vocab_xent_grad(x, w, target, dloss, want_dw=False, piece_bytes=bound)
        b = ll.vocab_xent_grad(x, w, target, dloss, want_dx=False, piece_bytes=bound)
        assert a[3] is None and b[2] is None
        _check(x, w, target, dloss, a, -100, "dx alone")
        _check(x, w, target, dloss, b, -100, "dw alone")
        assert torch.equal(both[0], a[0]) and torch.equal(both[0], b[0])
        f = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound,
                               dx=torch.empty((N, D), device="cuda"), dw=torch.empty((V, D + 5), device="cuda")[:, :D])
        assert f[2].dtype == f[3].dtype == torch.float32
        _check(x, w, target, dloss, f, -100, "fp32 gradients")


def test_rows_without_a_target_may_hold_anything():
    import torch
    ll = _ll()
    for N, V, D in ((20, 300, 64), (600, 2304, 128), (600, 2304, 192)):
        x, w, target, dloss = _case(N, V, D, "bfloat16", ignored=0.0)
        want = ll.vocab_xent_grad(x, w, torch.where(torch.arange(N, device="cuda") % 4 == 0, -100, target), dloss)
        bad = x.clone()
        bad[0::8] = float("nan")
        bad[4::8] = float("inf")
        t = target.clone()
        t[0::16] = -100
        t[4::16] = -1
        t[8::16] = V
        t[12::16] = 2 ** 40
        d = dloss.clone()
        d[0::4] = float("nan")
        got = ll.vocab_xent_grad(bad, w, t, d)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_all_rows_ignored_and_an_ignored_id_inside_the_vocabulary():
    import torch
    ll = _ll()
    x, w, target, dloss = _case(33, 500, 64, "float16", ignored=0.0)
    out = ll.vocab_xent_grad(x, w, torch.full_like(target, -100), dloss)
    for t in out:
        assert float(t.float().abs().max()) == 0
    target[3] = target[9] = 7
    out = ll.vocab_xent_grad(x, w, target, dloss, ignore_index=7)
    _check(x, w, target, dloss, out, 7, "ignore 7")
    assert float(out[0][3]) == 0 and float(out[0][9]) == 0


def test_no_rows():
    import torch
    ll = _ll()
    for dtype in (torch.bfloat16, torch.float16):
        x, w = torch.empty((0, 72), dtype=dtype, device="cuda"), torch.ones((700, 72), dtype=dtype, device="cuda")
        e = torch.empty(0, dtype=torch.int64, device="cuda")
        assert ll.vocab_xent(x, w, e)[0].shape == (0,)
        loss, lse, dx, dw = ll.vocab_xent_grad(x, w, e, torch.empty(0, device="cuda"), piece_bytes=1)
        assert dx.shape == (0, 72) and float(dw.float().abs().max()) == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_large_and_lopsided_logits(dtype):
    """Logits of hundreds (exp overflows without the maximum), a certain target
    (gradient near 0) and a hopeless one; entries of -inf (0 * exp)."""
    import torch
    ll = _ll()
    for N, V, D in ((12, 900, 64), (520, 2304, 64), (520, 2304, 192)):
        x, w, target, dloss = _case(N, V, D, dtype, std=30.0, ignored=0.1)
        _check(x, w, target, dloss, ll.vocab_xent_grad(x, w, target, dloss), -100, "large logits")
        best = (x.double() @ w.double().T).argmax(1)
        _check(x, w, best, dloss, ll.vocab_xent_grad(x, w, best, dloss), -100, "certain targets")
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    w = torch.zeros((600, 64), dtype=torch.bfloat16, device="cuda")
    w[100:, 0] = float("-inf")
    t = torch.tensor([0, 99, 50], device="cuda")
    for bound in (0, 1):  # a piece of -inf alone, too
        loss, lse = ll.vocab_xent(x, w, t, piece_bytes=bound)
        assert torch.allclose(lse, torch.full((3,), math.log(100.0), device="cuda"), rtol=1e-6)
        assert torch.equal(loss, lse)


def test_nan_stays_in_its_row():
    import torch
    ll = _ll()
    for N, V, D in ((9, 300, 64), (600, 2304, 128), (600, 2304, 192)):
        x, w, target, dloss = _case(N, V, D, "bfloat16", ignored=0.0)
        want = ll.vocab_xent_grad(x, w, target, dloss)
        bad = x.clone()
        bad[4, 5] = float("nan")
        got = ll.vocab_xent_grad(bad, w, target, dloss)
        keep = torch.arange(N, device="cuda") != 4
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[2][keep], want[2][keep])
        assert bool(got[0][4].isnan()) and bool(got[2][4].isnan().all())


def test_misaligned_operands():
    """x and w starting off 16-byte borders: copied, same values."""
    import torch
    ll = _ll()
    N, V, D = 50, 700, 64
    x, w, target, dloss = _case(N, V, D, "bfloat16")
    want = ll.vocab_xent_grad(x, w, target, dloss)
    mx = torch.empty(N * D + 1, dtype=x.dtype, device="cuda")[1:].view(N, D).copy_(x)
    mw = torch.empty(V * D + 3, dtype=x.dtype, device="cuda")[3:].view(V, D).copy_(w)
    got = ll.vocab_xent_grad(mx, mw, target, dloss)
    _check(x, w, target, dloss, got, -100, "misaligned")
    assert torch.allclose(got[0], want[0], rtol=1e-5, atol=1e-5)


def test_gradients_agree_with_differences():
    """sum(dloss * loss) by central differences in 64 bits of the definition."""
    import torch
    ll = _ll()
    g = _gen(3)
    N, V, D, step = 4, 11, 8, 1e-4
    x = torch.randn((N, D), generator=g, device="cuda").bfloat16()
    w = torch.randn((V, D), generator=g, device="cuda").bfloat16()
    target = torch.tensor([3, -100, 10, 0], device="cuda")
    dloss = torch.tensor([1.0, 2.0, 0.5, 1.5], device="cuda")
    _, _, dx, dw = ll.vocab_xent_grad(x, w, target, dloss, dx=torch.empty((N, D), device="cuda"),
                                      dw=torch.empty((V, D), device="cuda"))

    def f(xd, wd):
        z = xd @ wd.T
        at = target.clamp_min(0)[:, None]
        per = torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]
        return float((torch.where(target >= 0, per, 0.0) * dloss.double()).sum())

    h = _half(torch.bfloat16)
    for i, grad in enumerate((dx, dw)):
        for j in range(grad.numel()):
            plus, minus = [x.double(), w.double()], [x.double(), w.double()]
            plus[i].view(-1)[j] += step
            minus[i].view(-1)[j] -= step
            num = (f(*plus) - f(*minus)) / (2 * step)
            other = (w if i == 0 else x).double().abs().max().item()
            # |dz| sums to at most 2 |dloss| over a row, 5 over all rows; each rounded once
            assert abs(num - float(grad.view(-1)[j])) <= h * 10 * other + 1e-5


def test_streams_and_graph():
    import torch
    ll = _ll()
    for N, V, D, bound in ((30, 800, 72, 0), (1024, 4096, 128, 0), (512, 3000, 64, 4 << 20)):
        x, w, target, dloss = _case(N, V, D, "bfloat16")
        want = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
        torch.cuda.current_stream().wait_stream(side)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
        for _ in range(3):
            for t in got:
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for p, q in zip(got, want):
                assert torch.equal(p, q)
            torch.randn(64, 64, device="cuda").sum().item()
