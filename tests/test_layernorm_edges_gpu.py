"""Layer norm's gradient where mean * rstd is beyond fp32.

The rows are constant and given with their mean and a large rstd, so xhat is
0 and dx = rstd * (h - mean(h)), h = dy * gamma.  With u = 2^-24: a sum of D
terms in fp32 (D u of the sum of magnitudes), four roundings, half a step of
the stored type."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype,param", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32")])
@pytest.mark.parametrize("D", [1, 100, 101, 1000, 1001, 1800, 3001, 6000, 9001, 12001, 20000])
def test_lanes_past_the_rows_end_stay_out(D, dtype, param):
    """Widths that leave lanes without a column in every variant, whole chunks and parts of one."""
    import torch
    import recsys_linear_layers_amd as ll
    dt, g = getattr(torch, dtype), torch.Generator(device="cuda")
    g.manual_seed(D)
    N = 7
    x = torch.full((N, D), 1e20, device="cuda").to(dt)
    mean, rstd = x[:, 0].float().contiguous(), torch.full((N,), 1e20, device="cuda")
    dy = torch.randn((N, D), generator=g, device="cuda").to(dt)
    gamma = (1 + torch.rand(D, generator=g, device="cuda")).to(getattr(torch, param))
    dx, dgamma, dbeta = ll.layernorm_grad(dy, x, mean, rstd, gamma)
    h = dy.double() * gamma.double()
    r = rstd.double()[:, None]
    want = r * (h - h.mean(1, keepdim=True))
    half = torch.finfo(dt).eps / 2
    tol = r * (D + 8) * U * (h.abs() + h.abs().mean(1, keepdim=True)) + want.abs() * half * 1.01
    assert bool(((dx.double() - want).abs() <= tol).all())
    assert float(dgamma.float().abs().max()) == 0
    s, m = dy.double().sum(0), dy.double().abs().sum(0)
    assert bool(((dbeta.double() - s).abs() <= m * (N + 2) * U + s.abs() * torch.finfo(dbeta.dtype).eps / 2).all())
