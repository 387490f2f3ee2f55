"""The root-mean-square norm of rows and weights of any magnitude whose norm is of an
ordinary one: y = h * rstd * gamma passes through nothing larger or smaller than h, its
norm and y.  Powers of two, so that every step is exact and the results compare bit
for bit: rows of one magnitude 2^e, whose rstd is 2^-e (squares and their sum stay
between 2^-126 and 2^127, eps is 0), and y = +-gamma."""
import pytest

pytestmark = pytest.mark.gpu

# (columns, a row's magnitude, gamma's): h * gamma alone would be 2^132, or 2^-140 and less
CASES = [(4, 62, 70), (4, 62, 120), (3, -60, -80), (8, -60, -62), (256, 50, 100), (1000, 50, 90), (5003, -50, -100),
         (8192, 50, 80), (16384, 40, 120), (16640, 40, 100), (40000, -50, -110)]


@pytest.mark.parametrize("D,e,g", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small(D, e, g, dtype):
    import torch
    import recsys_linear_layers_amd as ll
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    sign = 1.0 - 2.0 * (torch.arange(D, device="cuda") % 3 == 1)
    n = D if D & (D - 1) == 0 else 1 << D.bit_length()  # a mean that is exact: zeros fill up to a power of two of columns
    rows = [sign * 2.0 ** e, sign.flip(0) * 2.0 ** (e - 1)]
    h = torch.stack([torch.nn.functional.pad(r, (0, n - D)) for r in rows])
    mean = (h.double() ** 2).mean(1)
    for pt in {dt, torch.float32}:
        gamma = torch.full((n,), 2.0 ** g, device="cuda").to(pt)
        y, kept, rstd = ll.rmsnorm(h.to(dt), gamma, eps=0.0)
        # rstd: a quotient and a root, each rounded once, and the mean exact: 2 u
        assert bool(((rstd.double() * mean.sqrt() - 1).abs() <= 2 * 2.0 ** -24).all())
        want = h * rstd[:, None]  # times a power of two: exact
        assert torch.equal(y, (want * 2.0 ** g).to(dt))
        q, scale, _, _ = ll.rmsnorm8(h.to(dt), gamma, eps=0.0)
        assert bool(torch.isfinite(scale).all()) and not bool(torch.isnan(q.float()).any())
        live = h != 0
        assert bool((q.float()[live].abs() == 448).all()) and bool((q.float()[~live] == 0).all())
