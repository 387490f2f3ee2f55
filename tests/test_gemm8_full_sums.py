"""The 8-bit product into a 16-bit C with sums of fp32's precision (full_sums), against 64 bits.

With S the sum of the terms' magnitudes and u = 2^-24, a sum is off by at most
(256 + blocks + 3 + 64) u S: a whole step (2 u) for each of a block's 128 additions, one
rounding for each block's fma, three for the scales' products, 64 for the partials of
a split K.  C's rounding comes once on top."""
import ctypes

import pytest

KINDS = ["FEW16x16", "FEW16x32", "FEW32x16", "FEW32x32", "FEW64x16", "FEW64x32", "TILE64x128", "TILE128x128",
         "TILE128x256", "TILE256x256"]


def _operand(rows, K, seed, dtype, squares):
    import torch
    import helpers8 as h
    x = h.normal((rows, K), seed) * torch.exp(h.normal((rows, 1), seed + 1))
    x[:, ::37] *= 50.0  # columns that stand out
    q, s = h.quantise(x, squares, dtype)
    buf = torch.full((rows, -(-K // 16) * 16), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:, :K] = q.view(torch.uint8).cuda()
    return buf.view(dtype)[:, :K], s.cuda()


def _check(got, a, sa, b, sb, squares):
    import torch
    import helpers8 as h
    A, B = h.dequantise(a, sa, False).cuda(), h.dequantise(b, sb, squares).cuda()
    ref, S = A @ B.T, A.abs() @ B.abs().T
    tol = ((256 + h.blocks(a.shape[1]) + 3 + 64) * h.U * S + ref.abs() * h.HALF_STEP[got.dtype] * (1 + 2 ** -10)
           + h.SMALL_STEP[got.dtype])
    # to nearest: what is half a step or more beyond the type's largest value becomes an infinity of its sign
    most = torch.finfo(got.dtype).max * (1 + h.HALF_STEP[got.dtype] / 2)
    beyond = torch.isinf(got)
    assert bool((ref.abs() + tol >= most)[beyond].all()) and bool((torch.sign(got) == torch.sign(ref))[beyond].all())
    assert bool(((got.double() - ref).abs() <= tol)[~beyond].all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [1, 3])
def test_every_kernel(monkeypatch, kind, splits):
    import torch
    import recsys_linear_layers_amd as ll
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    monkeypatch.setenv("LL_GEMM8_SPLITS", str(splits))
    M, N = (int(kind[3:5]) - 3, 333) if kind.startswith("FEW") else (261, 515)
    for K in (900, 1000):
        for squares in (True, False):
            a, sa = _operand(M, K, 1, torch.float8_e5m2 if squares else torch.float8_e4m3fn, False)
            b, sb = _operand(N, K, 3, torch.float8_e4m3fn, squares)
            full = ll.gemm8(a, sa, b, sb, out_dtype=torch.float32)
            for c in (torch.bfloat16, torch.float16):
                print(kind, splits, K, squares, c, flush=True)
                # the same sums in the same order, rounded once: fp32's, rounded
                got = ll.gemm8(a, sa, b, sb, out_dtype=c, full_sums=True)
                assert torch.equal(got, full.to(c))
                _check(got, a, sa, b, sb, squares)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 5003, 4099), (37, 500, 4099), (65, 127, 257), (128, 2000, 2048), (300, 260, 12),
                                   (511, 513, 515), (2500, 4100, 384)])
def test_as_chosen(M, N, K):
    import torch
    import recsys_linear_layers_amd as ll
    a, sa = _operand(M, K, 1, torch.float8_e4m3fn, False)
    b, sb = _operand(N, K, 3, torch.float8_e4m3fn, True)
    for c in (torch.bfloat16, torch.float16):
        buf = torch.full((M + 2, N + 5), 5.0, dtype=c, device="cuda")
        out = buf[1:M + 1, 3:N + 3]
        assert ll.gemm8(a, sa, b, sb, out=out, full_sums=True) is out
        _check(out, a, sa, b, sb, True)
        out.fill_(5.0)
        assert bool((buf == 5).all())
        assert torch.equal(ll.gemm8(a, sa, b, sb, out_dtype=torch.float32),
                           ll.gemm8(a, sa, b, sb, out_dtype=torch.float32, full_sums=True))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 50, 200, 600])
def test_small_products_beside_large_ones(M):
    """448 * 448 and 127 products of 1 in the first block, the large one's opposite in
    the second: 127 in full sums; without, all but what the large one's groups of
    eight drop, within 7 * 2^-13 of the magnitudes' sum."""
    import torch
    import recsys_linear_layers_amd as ll
    N, K, e4 = 300, 256, torch.float8_e4m3fn
    A, B = torch.ones(M, K), torch.ones(N, K)
    A[:, 0] = B[:, 0] = A[:, 128] = 448.0
    B[:, 128] = -448.0
    A[:, 129:] = 0.0
    a, b = A.to(e4).cuda(), B.to(e4).cuda()
    sa, sb = torch.ones(M, 2, device="cuda"), torch.ones(3, 2, device="cuda")
    for c in (torch.bfloat16, torch.float16):
        assert bool((ll.gemm8(a, sa, b, sb, out_dtype=c, full_sums=True) == 127).all())
        off = ll.gemm8(a, sa, b, sb, out_dtype=c).float() - 127
        assert bool((off.abs() <= 7 * 2.0 ** -13 * (2 * 448 ** 2 + 127)).all())


@pytest.mark.gpu
def test_empty_and_not_finite():
    import torch
    import recsys_linear_layers_amd as ll
    for M, N in ((5, 7), (200, 300)):
        a, b = (torch.empty((r, 0), dtype=torch.float8_e4m3fn, device="cuda") for r in (M, N))
        out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
        ll.gemm8(a, torch.ones(M, 0, device="cuda"), b, torch.ones(-(-N // 128), 0, device="cuda"), out=out,
                 full_sums=True)
        assert bool((out == 0).all())
    for M in (3, 400):
        a, sa = _operand(M, 300, 1, torch.float8_e4m3fn, False)
        b, sb = _operand(200, 300, 3, torch.float8_e4m3fn, True)
        sa[M // 2, 1] = float("nan")
        nan = torch.isnan(ll.gemm8(a, sa, b, sb, full_sums=True))
        assert bool(nan[M // 2].all()) and int(nan.sum()) == 200


@pytest.mark.gpu
def test_captured():
    """Replayed with the program's own work in between, the same bits each time; the
    sums' workspace belongs to the graph."""
    import torch
    import recsys_linear_layers_amd as ll
    for M in (40, 300):
        a, sa = _operand(M, 2000, 1, torch.float8_e4m3fn, False)
        b, sb = _operand(515, 2000, 3, torch.float8_e4m3fn, True)
        want = ll.gemm8(a, sa, b, sb, full_sums=True)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ll.gemm8(a, sa, b, sb, full_sums=True)
        for _ in range(3):
            out.fill_(0.5)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            torch.randn(300, 300, device="cuda").sum()
            torch.cuda.synchronize()


@pytest.mark.gpu
def test_c_of_more_elements_than_a_launch_takes():
    """The kernel that rounds the sums takes 1024 of a row per workgroup: 2^24 workgroups
    and more would be 2^32 threads, which a launch cannot have."""
    import torch
    import recsys_linear_layers_amd as ll
    M, N, K = 65600, 262144, 16
    if torch.cuda.mem_get_info()[0] < 8 * M * N:
        pytest.skip("C and its sums take 103 GB")
    g = torch.Generator().manual_seed(1)
    A, B = (torch.randint(-4, 5, (r, K), generator=g).float().cuda() for r in (M, N))
    a, b = A.to(torch.float8_e4m3fn), B.to(torch.float8_e4m3fn)
    out = torch.full((M, N), 77.5, dtype=torch.bfloat16, device="cuda")
    ll.gemm8(a, torch.ones(M, 1, device="cuda"), b, torch.ones(N // 128, 1, device="cuda"), out=out, full_sums=True)
    for m in range(0, M, 4096):
        want = A[m:m + 4096] @ B.T  # whole numbers up to 256: exact
        assert torch.equal(out[m:m + 4096], want.to(torch.bfloat16)), m
        del want
    del out
    torch.cuda.empty_cache()


def _desc(**kw):
    import recsys_linear_layers_amd as ll
    base = dict(M=200, N=300, K=256, stride_a=256, stride_b=256, stride_c=300, stride_am=1, stride_ab=200, stride_bn=2,
                stride_bb=1, a_type=ll.LL_E4M3, b_type=ll.LL_E4M3, c_type=ll.LL_BF16, b_block=128)
    base.update(kw)
    return ll.Gemm8Desc(**base)


def test_flags_and_workspace():
    """Unknown bits are refused; full sums of more than a few rows take their workspace."""
    import recsys_linear_layers_amd as ll
    P, Q, R, S, T = 4096, 1 << 30, 1 << 31, 3 << 30, 5 << 30
    for flags in (2, 3, 0x80000000):
        n = ctypes.c_size_t()
        assert ll._lib.gemm8_workspace_size(ctypes.byref(_desc(flags=flags)), ctypes.byref(n)) == ll.LL_ERR_INVALID_ARG
        assert ll._lib.gemm8_run(ctypes.byref(_desc(flags=flags)), P, Q, R, S, T, None, 0, None) == ll.LL_ERR_INVALID_ARG
        assert "flags" in ll.ll_last_error()
    full = ll.LL_GEMM8_FULL_SUMS
    assert ll.gemm8_workspace_size(_desc(flags=full)) >= 200 * 300 * 4
    assert ll.gemm8_workspace_size(_desc(flags=full, M=16)) == 0
    for kw in (dict(c_type=ll.LL_F32), dict(c_type=ll.LL_F32, M=16)):  # fp32 is full already
        assert ll.gemm8_describe(_desc(flags=full, **kw)) == ll.gemm8_describe(_desc(**kw))
    assert ll._lib.gemm8_run(ctypes.byref(_desc(flags=full)), P, Q, R, S, T, None, 0, None) == ll.LL_ERR_WORKSPACE
    assert ll._lib.gemm8_run(ctypes.byref(_desc(flags=full)), P, Q, R, S, T, T, 1 << 20, None) == ll.LL_ERR_INVALID_ARG
