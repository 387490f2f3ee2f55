"""Sizes whose row or column kernels would need more workgroups than one grid
may have (2^32 threads along x, 2^16 workgroups along y)."""
import pytest

from test_vocab_xent_gpu import _check

pytestmark = pytest.mark.gpu


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


def test_layernorm_gradient_of_2_to_27_columns():
    import torch
    ll = _ll()
    N, D = 2, 2 ** 27 + 64
    x = torch.tensor([[3.0], [5.0]], device="cuda").repeat(1, D)
    dy = torch.ones((N, D), device="cuda")
    dy[:, -1] = 2
    _, dgamma, dbeta = ll.layernorm_grad(dy, x, torch.zeros(N, device="cuda"), torch.ones(N, device="cuda"))
    assert bool((dgamma[:-1] == 8).all()) and bool((dbeta[:-1] == 2).all())
    assert float(dgamma[-1]) == 16 and float(dbeta[-1]) == 4


def _rows(N, V, D, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty((N, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.randn((V, D), generator=g, device="cuda").div_(D ** 0.5).bfloat16()
    return x, w, torch.randint(0, V, (N,), generator=g, device="cuda")


def _check_ends(x, w, target, what):
    """The first and the last thousand rows, with the tolerances of test_vocab_xent_gpu."""
    import torch
    dloss = torch.rand(len(target), device="cuda")
    loss, lse, dx, _ = _ll().vocab_xent_grad(x, w, target, dloss, want_dw=False)
    for rows in (slice(0, 1000), slice(len(target) - 1000, len(target))):
        _check(x[rows], w, target[rows], dloss[rows], (loss[rows], lse[rows], dx[rows], None), -100, what)


def test_loss_and_gradient_of_more_than_2_to_26_rows():
    x, w, target = _rows(2 ** 26 + 1000, 20, 8, 1)
    _check_ends(x, w, target, "narrow")


def test_softmax_in_the_product_of_more_than_2_to_22_rows():
    x, w, target = _rows(2 ** 22 + 1000, 300, 136, 2)
    assert "fused=1" in _ll().xent_plan_for(x, w, x).describe()
    _check_ends(x, w, target, "fused")
