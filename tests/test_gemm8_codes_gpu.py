"""Every value an 8-bit operand can hold, through every kernel of the product: taken one
at a time by a matrix of ones at single places, so that C holds the value itself."""
import pytest

pytestmark = pytest.mark.gpu
KINDS = [("FEW16x16", 16), ("FEW16x32", 16), ("FEW32x16", 32), ("FEW32x32", 32), ("FEW64x16", 64), ("FEW64x32", 64),
         ("TILE64x128", 256), ("TILE128x128", 256), ("TILE128x256", 256), ("TILE256x256", 256)]
E4, E5 = "float8_e4m3fn", "float8_e5m2"


def _codes(dtype):
    """[256] bytes, and those that stand for finite numbers."""
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    return codes, torch.isfinite(codes.view(getattr(torch, dtype)).float())


def _rounded(v, c):
    import torch
    return v.to(c) if c != torch.float32 else v


@pytest.mark.parametrize("kind,M", KINDS)
@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("squares", [True, False])
def test_finite_values_of_a(monkeypatch, kind, M, dtype, squares):
    """Row i of A holds the codes from i on; B picks them."""
    import torch
    import recsys_linear_layers_amd as ll
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    codes, finite = _codes(dtype)
    codes = codes[finite]
    K = 256
    at = (torch.arange(M)[:, None] * 16 + torch.arange(K)[None]) % len(codes)
    a = codes[at].cuda().view(getattr(torch, dtype))
    b = torch.eye(K).to(torch.float8_e4m3fn).cuda()
    sa, sb = torch.ones(M, 2, device="cuda"), torch.ones(2 if squares else K, 2, device="cuda")
    for c in (torch.bfloat16, torch.float16, torch.float32):
        for full in (False, True):
            assert torch.equal(ll.gemm8(a, sa, b, sb, out_dtype=c, full_sums=full), _rounded(a.float(), c)), (c, full)


@pytest.mark.parametrize("kind,M", KINDS)
@pytest.mark.parametrize("dtype", [E4, E5])
def test_finite_values_of_b(monkeypatch, kind, M, dtype):
    """The same for B (e4m3), picked by an A of either type."""
    import torch
    import recsys_linear_layers_amd as ll
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    codes, finite = _codes(E4)
    codes = codes[finite]
    K, N = 256, 300
    at = (torch.arange(N)[:, None] * 7 + torch.arange(K)[None]) % len(codes)
    b = codes[at].cuda().view(torch.float8_e4m3fn)
    a = torch.eye(K)[torch.arange(M) * 5 % K].to(getattr(torch, dtype)).cuda()
    want = b.float().t()[torch.arange(M).cuda() * 5 % K]
    sa, sb = torch.ones(M, 2, device="cuda"), torch.ones(N, 2, device="cuda")
    for c in (torch.bfloat16, torch.float16, torch.float32):
        for full in (False, True):
            assert torch.equal(ll.gemm8(a, sa, b, sb, out_dtype=c, full_sums=full), _rounded(want, c)), (c, full)


@pytest.mark.parametrize("kind,M", KINDS)
def test_infinities_and_nan(monkeypatch, kind, M):
    """They stay in their row of A or of B, with the sign that the sum has; the rest as
    if they were not there."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    N, K = 300, 300
    (a, sa), (a2, _) = (ll.quant8(h.normal((M, K), 1).cuda(), dtype=torch.float8_e5m2) for _ in range(2))
    (b, sb), (b2, _) = (ll.quant8(h.normal((N, K), 2).cuda(), squares=True) for _ in range(2))
    raw_a, raw_b = a2.view(torch.uint8), b2.view(torch.uint8)
    raw_a[1, 5], raw_a[2, 290], raw_a[3, 7] = 0x7C, 0xFC, 0x7F  # infinity, minus infinity, NaN
    raw_b[4, 150] = 0xFF
    for c in (torch.bfloat16, torch.float32):
        for full in (False, True):
            clean = ll.gemm8(a, sa, b, sb, out_dtype=c, full_sums=full)
            got = ll.gemm8(a2, sa, b2, sb, out_dtype=c, full_sums=full)
            bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
            bad[1:4] = True
            bad[:, 4] = True
            assert torch.equal(got[~bad], clean[~bad])
            assert bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[:, 4]).all())
            for row, k, sign in ((1, 5, 1.0), (2, 290, -1.0)):
                w = b.float()[:, k]
                want = torch.where(w == 0, float("nan"), sign * torch.sign(w) * float("inf"))
                want[4] = float("nan")
                assert torch.equal(torch.isnan(got[row].float()), torch.isnan(want)), (c, full, row)
                live = ~torch.isnan(want)
                assert torch.equal(got[row].float()[live], want[live]), (c, full, row)
