"""The product of quantised matrices against 64 bits.

With S the sum of the terms' magnitudes and u = 2^-24: a block's 128 products are
exact and added up in the matrix unit, at most a whole step (2 u) lost by each of
128 additions; the scales' product (two with row scales) and one fma per block
round once each, and so does each partial of a split K: (256 + blocks + 3 + 64) u S,
then C's rounding.  That is C in fp32, whose operands are widened.  The 8-bit
instruction of a 16-bit C also aligns each group of eight products to the largest,
P, and drops from the other seven what lies below 2^-13 of its power of two: 7
times less than 2^-13 P, and the groups' P add up to at most S."""
import pytest

pytestmark = pytest.mark.gpu


def _types():
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
            "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _operand(rows, K, seed, dtype, squares, pad=0):
    """A quantised matrix on the GPU, NaN bytes between its rows' ends and their stride."""
    import torch
    import helpers8 as h
    x = h.normal((rows, K), seed) * torch.exp(h.normal((rows, 1), seed + 1))
    q, s = h.quantise(x, squares, dtype)
    ld = -(-K // 16) * 16 + 16 * pad
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:, :K] = q.view(torch.uint8).cuda()
    s = s.cuda()
    return buf.view(dtype)[:, :K], s if squares else s.t().contiguous().t()


def _reference(a, sa, b, sb, squares):
    import helpers8 as h
    A, B = h.dequantise(a, sa, False).cuda(), h.dequantise(b, sb, squares).cuda()
    return A @ B.T, A.abs() @ B.abs().T


def _check(got, ref, S, K):
    import torch
    import helpers8 as h
    aligned = 0.0 if got.dtype == torch.float32 else 7 * 2.0 ** -13
    tol = ((256 + h.blocks(K) + 3 + 64) * h.U + aligned) * S + ref.abs() * h.HALF_STEP[got.dtype] * (1 + 2 ** -10) + h.SMALL_STEP[got.dtype]
    # a value that rounds beyond the type's largest is infinite: half a step above it
    most = torch.finfo(got.dtype).max * (1 + h.HALF_STEP[got.dtype] / 2)
    beyond = torch.isinf(got)
    assert not bool(torch.isnan(got).any()) and bool((ref.abs() + tol >= most)[beyond].all())
    assert bool((torch.sign(got) == torch.sign(ref))[beyond].all())
    off = torch.where(beyond, 0.0, (got.double() - ref).abs()) - tol
    assert bool((off <= 0).all()), (off.max().item(), (off > 0).sum().item())


SHAPES = [(1, 64, 64), (1, 1, 1), (1, 5003, 4099), (2, 130, 127), (7, 1000, 128), (16, 16, 129), (16, 257, 1040),
          (17, 300, 8192), (31, 33, 40), (32, 512, 4096), (33, 129, 300), (37, 5003, 4099), (64, 1024, 2048),
          (64, 31, 20000), (65, 127, 257), (100, 700, 1000), (128, 128, 128), (129, 300, 5000), (200, 4000, 264),
          (256, 256, 1024), (511, 513, 515), (1000, 136, 33), (300, 260, 12), (2500, 4100, 384), (4096, 2570, 200)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("squares", [True, False])
def test_against_64_bits(M, N, K, squares):
    import recsys_linear_layers_amd as ll
    t = _types()
    qa = t["e5m2"] if (M + N) % 3 == 0 else t["e4m3"]
    a, sa = _operand(M, K, 1, qa, False, pad=M % 2)
    b, sb = _operand(N, K, 3, t["e4m3"], squares, pad=N % 2)
    ref, S = _reference(a, sa, b, sb, squares)
    for c in ("bf16", "f16", "f32"):
        print(M, N, K, squares, c, flush=True)
        _check(ll.gemm8(a, sa, b, sb, out_dtype=t[c]), ref, S, K)


@pytest.mark.parametrize("kind,M,N,K", [
    ("FEW16x16", 3, 100, 300), ("FEW16x16", 16, 515, 5000), ("FEW16x32", 9, 333, 1000), ("FEW16x32", 1, 70, 9000),
    ("FEW32x16", 30, 100, 130), ("FEW32x16", 17, 90, 7000), ("FEW32x32", 32, 64, 64), ("FEW32x32", 5, 200, 4100),
    ("FEW64x16", 64, 64, 64), ("FEW64x16", 40, 333, 3000), ("FEW64x32", 9, 333, 1000), ("FEW64x32", 64, 95, 3000),
    ("TILE64x128", 3, 100, 300), ("TILE64x128", 64, 257, 5000), ("TILE64x128", 130, 60, 1030),
    ("TILE128x128", 3, 100, 300), ("TILE128x128", 300, 200, 700), ("TILE128x128", 129, 385, 4100),
    ("TILE128x256", 5, 70, 90), ("TILE128x256", 200, 300, 3000), ("TILE128x256", 129, 513, 1111),
    ("TILE256x256", 5, 70, 90), ("TILE256x256", 300, 520, 1000), ("TILE256x256", 513, 257, 4100)])
@pytest.mark.parametrize("splits", [1, 3])
def test_every_kernel_and_split(monkeypatch, kind, M, N, K, splits):
    """Kernels and splits that the sizes alone would not pick."""
    import recsys_linear_layers_amd as ll
    t = _types()
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    monkeypatch.setenv("LL_GEMM8_SPLITS", str(splits))
    for squares in (True, False):
        a, sa = _operand(M, K, 1, t["e4m3"], False)
        b, sb = _operand(N, K, 3, t["e4m3"], squares)
        ref, S = _reference(a, sa, b, sb, squares)
        for c in ("bf16", "f32"):
            out = a.new_empty((M, N), dtype=t[c])
            assert f"kernel={kind} " in ll.gemm8_describe(ll.gemm8_desc_for(a, sa, b, sb, out))
            _check(ll.gemm8(a, sa, b, sb, out=out), ref, S, K)


@pytest.mark.parametrize("kind,M", [("FEW16x16", 16), ("FEW16x32", 5), ("FEW32x16", 31), ("FEW32x32", 32), ("FEW64x16", 64),
                                    ("FEW64x32", 37), ("FEW64x32", 64)])
@pytest.mark.parametrize("K", [100, 128, 1000, 2100, 3456])
def test_rows_of_whole_lines(monkeypatch, kind, M, K):
    """Rows at multiples of 128 bytes, from a line's start and from behind it, K ending anywhere: the same bits."""
    import torch
    import recsys_linear_layers_amd as ll
    t = _types()
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    ld = -(-K // 128) * 128 + 128
    for N, squares in ((333, True), (65, False)):
        a, sa = _operand(M, K, 1, t["e5m2"] if squares else t["e4m3"], False)
        b, sb = _operand(N, K, 3, t["e4m3"], squares)
        ref, S = _reference(a, sa, b, sb, squares)
        for c in ("bf16", "f32"):
            got = []
            for start in (0, 16):
                near = []
                for x in (a, b):
                    buf = torch.full((len(x) * ld + 128,), 0x7F, dtype=torch.uint8, device="cuda")
                    buf = buf[start:start + len(x) * ld].view(len(x), ld)
                    buf[:, :K] = x.view(torch.uint8)
                    near.append(buf.view(x.dtype)[:, :K])
                got.append(ll.gemm8(near[0], sa, near[1], sb, out_dtype=t[c]))
                _check(got[-1], ref, S, K)
            assert torch.equal(got[0], got[1])


@pytest.mark.parametrize("kind,bm,bn", [("TILE64x128", 64, 128), ("TILE128x128", 128, 128), ("TILE128x256", 128, 256),
                                        ("TILE256x256", 256, 256)])
@pytest.mark.parametrize("K", [20, 128, 260, 1000])
def test_more_tiles_than_compute_units(monkeypatch, kind, bm, bn, K):
    """Workgroups that take several tiles, of one step each and of several, in 9 rows of
    tiles (a group of 8 and a row alone), with short last pieces of K at each tile's end."""
    import recsys_linear_layers_amd as ll
    t = _types()
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    monkeypatch.setenv("LL_GEMM8_SPLITS", "1")
    M, N = 9 * bm - 5, 61 * bn - 3
    for squares in (True, False):
        a, sa = _operand(M, K, 1, t["e5m2"] if squares else t["e4m3"], False, pad=1)
        b, sb = _operand(N, K, 3, t["e4m3"], squares)
        ref, S = _reference(a, sa, b, sb, squares)
        for c in ("bf16", "f16", "f32"):
            _check(ll.gemm8(a, sa, b, sb, out_dtype=t[c]), ref, S, K)


@pytest.mark.parametrize("kind,M,N", [
    ("FEW16x16", 3, 333), ("FEW16x32", 16, 333), ("FEW32x16", 31, 333), ("FEW32x32", 20, 333), ("FEW64x16", 64, 333),
    ("FEW64x32", 50, 333), ("TILE64x128", 133, 259), ("TILE128x128", 261, 259), ("TILE128x256", 261, 515),
    ("TILE256x256", 517, 515)])
@pytest.mark.parametrize("qa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("squares", [True, False])
def test_every_variant(monkeypatch, kind, M, N, qa, squares):
    """Each instantiation, with one to five blocks for each of eight waves, whole lines and not, a short block and none."""
    import recsys_linear_layers_amd as ll
    t = _types()
    monkeypatch.setenv("LL_GEMM8_KIND", kind)
    monkeypatch.setenv("LL_GEMM8_SPLITS", "1")
    for K, pad in ((900, 7), (1900, 1), (3333, 2), (3333, 7), (4100, 0), (4100, 7), (4096, 0), (4096, 1)):
        a, sa = _operand(M, K, 1, t[qa], False, pad=pad)
        b, sb = _operand(N, K, 3, t["e4m3"], squares, pad=pad)
        ref, S = _reference(a, sa, b, sb, squares)
        for c in ("bf16", "f16", "f32"):
            _check(ll.gemm8(a, sa, b, sb, out_dtype=t[c]), ref, S, K)


def test_integers_are_exact():
    """Small whole numbers with scales of 2 and 1/2: every product is at least 2^-4 of
    any other, every sum exact in fp32, and C that sum rounded once."""
    import torch
    import recsys_linear_layers_amd as ll
    g = torch.Generator().manual_seed(1)
    e4 = _types()["e4m3"]
    for M, N, K in ((1, 300, 500), (20, 40, 3000), (70, 200, 1111), (600, 800, 640), (3000, 2600, 300)):
        A = torch.randint(-4, 5, (M, K), generator=g).double()
        B = torch.randint(-4, 5, (N, K), generator=g).double()
        ld = -(-K // 16) * 16
        a, b = (torch.zeros((len(v), ld), dtype=torch.uint8, device="cuda").view(e4)[:, :K] for v in (A, B))
        a.copy_(A.float().to(e4).cuda())
        b.copy_(B.float().to(e4).cuda())
        kb = -(-K // 128)
        sa = torch.full((M, kb), 2.0, device="cuda")
        for rows in (N, -(-N // 128)):
            sb = torch.full((rows, kb), 0.5, device="cuda")
            want = A.cuda() @ B.cuda().T
            for c in (torch.float32, torch.bfloat16, torch.float16):
                assert torch.equal(ll.gemm8(a, sa, b, sb, out_dtype=c), want.to(c)), (M, N, K, rows, c)


@pytest.mark.parametrize("M", [1, 20, 50, 200, 1500])
def test_rows_beyond_c_and_scale_strides(M):
    """A C inside a larger buffer at any alignment leaves its surroundings alone;
    scales of any strides."""
    import torch
    import recsys_linear_layers_amd as ll
    t = _types()
    N, K = 1301, 700
    a, sa = _operand(M, K, 1, t["e4m3"], False)
    b, sb = _operand(N, K, 3, t["e4m3"], False)
    want = {c: ll.gemm8(a, sa, b, sb, out_dtype=t[c]) for c in ("bf16", "f32")}
    for c in ("bf16", "f32"):
        for ld, off in ((N, 0), (N + 3, 1), (N + 11, 8), (1312, 4)):
            buf = torch.full(((M + 2) * ld + off,), 5.0, dtype=t[c], device="cuda")
            out = buf[off:off + (M + 2) * ld].view(M + 2, ld)[1:M + 1, :N]
            ll.gemm8(a, sa, b, sb, out=out)
            assert torch.equal(out, want[c])
            out.fill_(5.0)
            assert bool((buf == 5).all())
    kb = sa.shape[1]
    for shape in (lambda s: s.contiguous(), lambda s: torch.stack([s, s], 2)[:, :, 1],
                  lambda s: torch.cat([s, s], 0)[: s.shape[0]]):
        assert torch.equal(ll.gemm8(a, shape(sa), b, shape(sb)), want["bf16"])


@pytest.mark.parametrize("M,N", [(1, 400), (40, 400), (100, 400), (400, 300), (2600, 4100)])
def test_not_finite_stays_in_its_rows(M, N):
    """A row of A with a NaN scale gives a row of NaN, a block of B its columns; the
    rest is as if they were zero."""
    import torch
    import recsys_linear_layers_amd as ll
    t = _types()
    K = 500
    for squares in (True, False):
        a, sa = _operand(M, K, 1, t["e4m3"], False)
        b, sb = _operand(N, K, 3, t["e4m3"], squares)
        clean = ll.gemm8(a, sa, b, sb)
        sa[M // 2, 1] = float("nan")
        sb[1, 2] = float("nan")
        got = ll.gemm8(a, sa, b, sb)
        bad_rows = torch.zeros(M, 1, dtype=torch.bool, device="cuda")
        bad_rows[M // 2] = True
        bad = torch.zeros(1, N, dtype=torch.bool, device="cuda")
        bad[:, slice(128, 256) if squares else slice(1, 2)] = True
        assert torch.equal(torch.isnan(got), (bad_rows | bad).expand(M, N))
        assert torch.equal(got[~torch.isnan(got)], clean[~torch.isnan(got)])


def test_empty():
    import torch
    import recsys_linear_layers_amd as ll
    e4 = _types()["e4m3"]
    for M, N, K in ((0, 5, 32), (5, 0, 32), (5, 7, 0), (200, 300, 0)):
        a, b = torch.empty((M, K), dtype=e4, device="cuda"), torch.empty((N, K), dtype=e4, device="cuda")
        kb = -(-K // 128)
        out = torch.full((M, N), 3.0, device="cuda")
        ll.gemm8(a, torch.ones(M, kb, device="cuda"), b, torch.ones(-(-N // 128), kb, device="cuda"), out=out)
        assert bool((out == 0).all())


def test_equal_bits_and_a_workspace_of_any_content():
    import torch
    import recsys_linear_layers_amd as ll
    t = _types()
    a, sa = _operand(100, 5000, 1, t["e4m3"], False)
    b, sb = _operand(300, 5000, 3, t["e4m3"], True)
    out = torch.empty((100, 300), device="cuda")
    desc = ll.gemm8_desc_for(a, sa, b, sb, out)
    need = ll.gemm8_workspace_size(desc)
    assert need > 0
    first = None
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        ll.gemm8_run(desc, a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), out.data_ptr(), ws.data_ptr(), need)
        got = out.clone()
        first = got if first is None else first
        assert torch.equal(first, got)


def test_long_k():
    import recsys_linear_layers_amd as ll
    t = _types()
    for M, N, K in ((3, 40, 300000), (140, 150, 100003)):
        a, sa = _operand(M, K, 1, t["e4m3"], False)
        b, sb = _operand(N, K, 3, t["e4m3"], True)
        ref, S = _reference(a, sa, b, sb, True)
        _check(ll.gemm8(a, sa, b, sb, out_dtype=t["f32"]), ref, S, K)
