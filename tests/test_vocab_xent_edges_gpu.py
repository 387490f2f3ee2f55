"""The cross entropy where values are at the ends of their types' ranges, with the
tolerances of test_vocab_xent_gpu."""
import pytest

from test_vocab_xent_gpu import _case, _check, _ll

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 100])
def test_a_row_without_a_target_has_no_gradient_beside_huge_entries(D):
    """Narrow rows: the sum over w itself, which such a row meets, is beyond fp32 here."""
    import torch
    ll = _ll()
    N, V = 300, 5003
    x, w, target, dloss = _case(N, V, D, "bfloat16", ignored=0.3)
    assert ll.xent_plan_for(x, w, x.clone(), w.clone()).describe().startswith("narrow")
    w[:, 1] = -3e38
    x[:, 1] = 0
    dead = target < 0
    for dx in (torch.empty_like(x), torch.empty((N, D), device="cuda")):
        out = ll.vocab_xent_grad(x, w, target, dloss, dx=dx)
        assert 0 < int(dead.sum()) < N and bool((dx[dead] == 0).all())
        assert bool(torch.isfinite(out[0]).all()) and bool(torch.isfinite(dx[:, 2:]).all())


# Entries of the vocabulary masked by huge negative logits, and logits far above
# all others: x has a column of ones, and the same column of w holds the mask or
# the far value, so the products are exact where they are large.
# path, rows, entries, width, bound of a piece
PATHS = [("fused=1", 600, 20000, 192, 0), ("fused=1", 600, 20000, 192, 4 * 1024 * 768 * 2), ("fused=1", 2000, 9001, 136, 1),
         ("narrow", 300, 5003, 64, 0), ("few_rows", 20, 5003, 200, 0), ("fused=0", 100, 9000, 192, 0),
         ("fused=0", 100, 40000, 136, 0)]


def _run(path, N, V, D, bound, dtype, far, at):
    import torch
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, seed=11)
    x[:, 0] = 1
    w[:, 0] = 0
    w[at, 0] = far
    plan = ll.xent_plan_for(x, w, x.clone(), w.clone(), piece_bytes=bound).describe()
    assert path in plan, plan
    what = f"{dtype} {path} {N}x{V}x{D} {far:g}"
    if far < 0:  # no row's target is a masked entry
        live = torch.ones(V, dtype=torch.bool, device="cuda")
        live[at] = False
        keep = torch.nonzero(live).squeeze(1)
        target = torch.where(target >= 0, keep[target.clamp_min(0) % len(keep)], target)
    else:
        target[::3] = torch.where(target[::3] >= 0, at.start, target[::3])
    loss, lse = ll.vocab_xent(x, w, target, piece_bytes=bound)
    _check(x, w, target, None, (loss, lse, None, None), -100, what)
    out = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
    _check(x, w, target, dloss, out, -100, what)
    if far < 0:
        assert float(out[3][at].float().abs().max()) == 0, "a masked entry has a gradient"


@pytest.mark.parametrize("path,N,V,D,bound", PATHS)
@pytest.mark.parametrize("dtype,mask", [("bfloat16", -3.3895e38), ("bfloat16", -1e30), ("bfloat16", -1e9), ("bfloat16", -1e5),
                                        ("float16", -65504.0)])
def test_masked_entries(path, N, V, D, bound, dtype, mask):
    """A third of the vocabulary masked: whole blocks of 128 columns, and parts of two more."""
    _run(path, N, V, D, bound, dtype, mask, slice(V // 3 + 5, 2 * V // 3))


@pytest.mark.parametrize("path,N,V,D,bound", PATHS)
@pytest.mark.parametrize("dtype,far", [("bfloat16", 1e30), ("bfloat16", 1e9), ("bfloat16", 3e4), ("float16", 3e4)])
def test_one_entry_far_above_the_others(path, N, V, D, bound, dtype, far):
    _run(path, N, V, D, bound, dtype, far, slice(V // 2, V // 2 + 1))


@pytest.mark.parametrize("path,N,V,D,bound", PATHS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_the_loss_of_a_certain_target_is_not_negative(path, N, V, D, bound, dtype):
    """Targets that have all of the probability but what rounds away: the loss is
    zero or more, as it is in exact arithmetic."""
    import torch
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, seed=12, std=40.0)
    live = target >= 0
    target = torch.where(live, (x.double() @ w.double().T).argmax(1), target)
    assert path in ll.xent_plan_for(x, w, x.clone(), w.clone(), piece_bytes=bound).describe()
    loss, lse = ll.vocab_xent(x, w, target, piece_bytes=bound)
    assert bool((loss >= 0).all()), loss.min()
    out = ll.vocab_xent_grad(x, w, target, dloss, piece_bytes=bound)
    assert bool((out[0] >= 0).all()), out[0].min()
    _check(x, w, target, dloss, out, -100, f"{dtype} {path}")


@pytest.mark.parametrize("path,N,V,D,bound", PATHS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_entries_masked_by_minus_infinity(path, N, V, D, bound, dtype):
    """Loss and dw (dx meets 0 times infinity by its formula) as with a mask of -6e4, rows without a target among them."""
    import torch
    ll = _ll()
    x, w, target, dloss = _case(N, V, D, dtype, seed=13, ignored=0.3)
    at = slice(V // 3 + 5, 2 * V // 3)
    x[:, 0] = 1
    w[:, 0] = 0
    target = torch.where((target >= at.start) & (target < at.stop), 3, target)
    finite, endless = w.clone(), w.clone()
    finite[at, 0], endless[at, 0] = -6e4, float("-inf")
    assert path in ll.xent_plan_for(x, w, None, w.clone(), piece_bytes=bound).describe()
    loss, lse, _, dw = ll.vocab_xent_grad(x, endless, target, dloss, want_dx=False, piece_bytes=bound)
    _check(x, finite, target, dloss, (loss, lse, None, dw), -100, f"{dtype} {path}")
    assert float(dw[at].float().abs().max()) == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_a_far_row_leaves_the_others_as_they_are(dtype):
    """One row of every sixteen with logits of thousands: the other rows' bits, with and without it."""
    import torch
    ll = _ll()
    for bound in (0, 1):
        x, w, target, dloss = _case(600, 20000, 192, dtype, seed=14, ignored=0.1)
        assert "fused=1" in ll.xent_plan_for(x, w, x, piece_bytes=bound).describe()
        far = x.clone()
        far[5::16] *= 1000
        keep = torch.arange(600, device="cuda") % 16 != 5
        a, b = (ll.vocab_xent_grad(p, w, target, dloss, want_dw=False, piece_bytes=bound) for p in (x, far))
        assert all(torch.equal(p[keep], q[keep]) for p, q in zip(a[:3], b[:3]))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_what_the_workspace_holds_does_not_matter(dtype):
    """Rows up to whole tiles, columns up to whole parts: nothing is read there that the call has not written.
    The workspace is filled with large numbers, NaN and zeros in turn."""
    import torch
    ll = _ll()
    for N, V, D, bound in ((382, 20000, 304, 1 << 22), (2418, 3434, 192, 1), (777, 5003, 200, 0), (130, 40000, 136, 0),
                           (20, 5003, 200, 0), (300, 5003, 64, 0), (100, 9000, 192, 1)):
        x, w, target, dloss = _case(N, V, D, dtype, seed=15)
        plan = ll.xent_plan_for(x, w, x, w, piece_bytes=bound)
        outs = []
        for fill in (1e30, float("nan"), 0.0, -1e9):
            ws = torch.full((plan.ws_bytes // 4,), fill, device="cuda")
            loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
            dx, dw = torch.empty_like(x), torch.empty_like(w)
            ll.xent_run(plan.handle, x.data_ptr(), w.data_ptr(), target.data_ptr(), dloss.data_ptr(), loss.data_ptr(),
                        lse.data_ptr(), dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), plan.ws_bytes,
                        torch.cuda.current_stream().cuda_stream)
            outs.append((loss, lse, dx, dw))
        for out in outs[1:]:
            assert all(torch.equal(p, q) for p, q in zip(out, outs[0])), (N, V, D, bound)
