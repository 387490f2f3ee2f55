"""The cross entropy where values are at the ends of their types' ranges."""
import pytest

from test_vocab_xent_gpu import _case, _ll

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
