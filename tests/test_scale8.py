"""A quantised block's scale, max(amax / F, 2^-126), and its reciprocal are the correctly
rounded ones, for every fp32 amax there is: both are formed without a division.

The divisions here are in 64 bits, rounded to fp32 afterwards.  A quotient of two
numbers of 24 bits is never so near the middle of two of 24 that 53 bits would
hide on which side it lies (53 >= 2 * 24 + 2), so that is the correctly rounded fp32
quotient (below 2^-126, where fp32 has fewer bits, the maximum takes over)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LARGEST = {3: 448.0, 4: 57344.0}


def _check():
    lib = ctypes.CDLL(os.path.join(ROOT, "recsys_linear_layers_amd", "libllprobes.so"))
    lib.ll_check_scale8.argtypes = [ctypes.c_int, ctypes.c_uint32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p]
    return lib.ll_check_scale8


def test_refusals():
    f = _check()
    assert f(2, 0, 16, 4096, 8192, None) == -1
    assert f(3, 0, -1, 4096, 8192, None) == -1
    assert f(3, 1 << 31, 1, 4096, 8192, None) == -1
    assert f(3, 1, 1 << 31, 4096, 8192, None) == -1
    assert f(3, 0, 16, None, 8192, None) == -1 and f(3, 0, 16, 4096, 8194, None) == -1
    assert f(4, 0, 0, None, None, None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q", [3, 4])
def test_every_amax(q):
    import torch
    f, step, end = _check(), 1 << 26, 0x7F800000  # up to infinity's pattern
    scale, inv = torch.empty(step, device="cuda"), torch.empty(step, device="cuda")
    F = torch.full((1,), LARGEST[q], dtype=torch.float64, device="cuda")  # a number would make it a product
    seen = 0
    for first in range(0, end, step):
        n = min(step, end - first)
        assert f(q, first, n, scale.data_ptr(), inv.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        amax = torch.arange(first, first + n, dtype=torch.int32, device="cuda").view(torch.float32)
        want = (amax.double() / F).clamp_min(2.0 ** -126).float()
        assert torch.equal(scale[:n], want), hex(first)
        assert torch.equal(inv[:n], (1.0 / want.double()).float()), hex(first)
        seen += n
    assert seen == end
    # infinity and every NaN
    n = 1 << 23
    assert f(q, end, n, scale.data_ptr(), inv.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert bool(torch.isnan(scale[:n]).all()) and bool(torch.isnan(inv[:n]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("q,exponents", [("e4m3", (9, 127, 254)), ("e5m2", (16, 127, 254))])
def test_every_mantissa_through_quant8(q, exponents):
    """Columns of one value: every mantissa at the smallest scale's edge (F * 2^-126), at 1 and at the top."""
    import torch
    import recsys_linear_layers_amd as ll
    dtype, code = {"e4m3": (torch.float8_e4m3fn, 3), "e5m2": (torch.float8_e5m2, 4)}[q]
    F = torch.full((1,), LARGEST[code], dtype=torch.float64, device="cuda")
    for e in exponents:
        first = e << 23
        x = torch.arange(first, first + (1 << 23), dtype=torch.int32, device="cuda").view(torch.float32)[:, None]
        v, scale = ll.quant8(x, dtype=dtype)
        want = (x.double() / F).clamp_min(2.0 ** -126).float()
        assert torch.equal(scale, want), e
        # at most F (1 + 2^-22) before it is rounded, and at least F / 2 at the edge: within half a step
        assert bool(((v.double() * scale.double() - x.double()).abs()
                     <= x.double() * 2.0 ** (-4 if q == "e4m3" else -3)).all())
