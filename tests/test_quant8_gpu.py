"""Quantisation in blocks of 128 against the definition, bit for bit, and its
error against 64 bits."""
import pytest

pytestmark = pytest.mark.gpu


def _types():
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
            "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _check(x, got, squares, dtype):
    """got: (q, scale) for x on the host."""
    import torch
    import helpers8 as h
    q, scale = got
    want_q, want_s = h.quantise(x, squares, dtype)
    assert q.dtype == dtype and q.shape == x.shape and scale.shape == want_s.shape
    assert torch.equal(torch.isnan(scale.cpu()), torch.isnan(want_s))
    assert torch.equal(torch.nan_to_num(scale.cpu()), torch.nan_to_num(want_s))
    assert h.same_bytes(q, want_q)


@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (1, 128, 0), (1, 8192, 0), (3, 127, 1), (128, 128, 0), (129, 257, 3),
                                     (127, 1000, 5), (300, 130, 8), (8, 5003, 3), (1000, 17, 0), (513, 640, 0)])
@pytest.mark.parametrize("type_", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("squares", [False, True])
def test_every_form(n, d, pad, type_, squares):
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    t = _types()
    q8 = t["e5m2"] if (n + d) % 3 == 0 else t["e4m3"]
    x = h.normal((n, d), 7 * n + d, t[type_], 3.0)
    x[n // 2] *= 100.0
    x[:, d // 2] *= 0.01
    dev = h.strided(x, pad)
    q, s, qt, st = ll.quant8_pair(dev, squares=squares, dtype=q8)
    _check(x, (q, s), squares, q8)
    _check(x.t(), (qt, st), squares, q8)
    _check(x, ll.quant8(dev, squares=squares, dtype=q8), squares, q8)
    _check(x.t(), ll.quant8(dev, squares=squares, dtype=q8, transpose=True), squares, q8)
    assert q.stride(0) % 16 == 0 and qt.stride(0) % 16 == 0


def test_error_is_half_a_step():
    """q * scale against x in 64 bits: 1/scale, the product and the rounding to 8
    bits are off by 2^-24, 2^-24 and half a step, below the smallest normal number
    half its distance."""
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    for q8 in (_types()["e4m3"], _types()["e5m2"]):
        x = h.normal((200, 700), 5) * 10.0 ** h.normal((200, 700), 6)
        q, s = ll.quant8(x.cuda(), dtype=q8)
        err = (h.dequantise(q, s, False) - x.double()).abs()
        bound = x.double().abs() * (h.HALF_STEP[q8] + 3 * h.U) + h.expand(s.cpu().double(), 200, 700, False) * h.SMALL_STEP[q8] * (1 + 4 * h.U)
        assert bool((err <= bound).all())


@pytest.mark.parametrize("squares", [False, True])
def test_extremes(squares):
    """Blocks of zeros, of denormals, of the type's largest values, with a NaN or an
    infinity: a block that is not finite is NaN, its neighbours are not."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    x = h.normal((256, 512), 3)
    x[0:128, 0:128] = 0.0
    x[0:128, 128:256] *= 1e-42
    x[0:128, 256:384] = 3.4e38
    x[0:128, 384:512] *= 1e-37
    x[130, 5] = float("nan")
    x[200, 300] = float("inf")
    x[255, 511] = -float("inf")
    for q8 in (_types()["e4m3"], _types()["e5m2"]):
        q, s, qt, st = ll.quant8_pair(x.cuda(), squares=squares, dtype=q8)
        _check(x, (q, s), squares, q8)
        _check(x.t(), (qt, st), squares, q8)
        assert bool(torch.isnan(s).any()) and bool(torch.isfinite(s).any())
        assert bool((q.cpu().float()[0:128, 0:128] == 0).all())


def test_nothing_past_the_rows_is_written():
    """The bytes between the rows' ends and the stride, and the rows behind."""
    import torch
    import recsys_linear_layers_amd as ll
    import helpers8 as h
    n, d = 130, 201
    x = h.normal((n, d), 9).cuda()
    buf = torch.full((n + 2, 256), 0x5A, dtype=torch.uint8, device="cuda")
    buft = torch.full((d + 2, 256), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((n + 2, 5), 7.0, device="cuda")
    st = torch.full((d + 2, 5), 7.0, device="cuda")
    desc = ll.Quant8Desc(n, d, d, 256, 256, 5, 2, 5, 2, ll.LL_F32, ll.LL_E4M3, 1)
    ll.quant8_run(desc, x.data_ptr(), buf.data_ptr(), s.data_ptr(), buft.data_ptr(), st.data_ptr())
    torch.cuda.synchronize()
    assert bool((buf[n:] == 0x5A).all()) and bool((buf[:, d:] == 0x5A).all())
    assert bool((buft[d:] == 0x5A).all()) and bool((buft[:, n:] == 0x5A).all())
    assert bool((s[n:] == 7).all()) and bool((s[:, 1::2] == 7).all()) and bool((s[:n, 4] == 7).all())
    want, ws = h.quantise(x.cpu(), False, _types()["e4m3"])
    assert h.same_bytes(buf[:n, :d].view(_types()["e4m3"]), want) and torch.equal(s[:n, 0:3:2].cpu(), ws)


def test_empty():
    import torch
    import recsys_linear_layers_amd as ll
    for n, d in ((0, 5), (5, 0), (0, 0)):
        q, s, qt, st = ll.quant8_pair(torch.empty(n, d, device="cuda"))
        assert q.shape == (n, d) and qt.shape == (d, n) and s.shape == (n, -(-d // 128))
