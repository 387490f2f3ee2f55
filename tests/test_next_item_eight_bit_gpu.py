"""The example's hidden layer in 8 bits: product, bias and relu rounded once, as in 16 bits."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("width,hidden,rows", [(64, 96, 30), (200, 264, 700)])
def test_hidden_layer_is_rounded_once(width, hidden, rows):
    """Biases the size of the products, so that many sums are far smaller than their
    terms.  With S the magnitudes' sum and u = 2^-24: (256 + blocks + 2) u S for the
    product, u of the sum for the bias's addition (at most u (S + |b|)), and one rounding
    to bf16."""
    import helpers8 as h
    import torch
    spec = importlib.util.spec_from_file_location("next_item_bias", os.path.join(ROOT, "examples", "next_item.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    model = ex.NextItem(301, width, hidden, seed=3, eight_bit=True)
    model.master["b1"].copy_(h.normal((hidden,), 5))
    model.refresh()
    _, (n8, got, _) = model.middle(h.normal((rows, width), 6, torch.bfloat16).cuda())
    A, B = h.dequantise(*n8[:2], False), h.dequantise(*model.w8["W1"][:2], True)
    b = model.w["b1"].double().cpu()
    product, S = A @ B.T, A.abs() @ B.abs().T
    want = torch.relu(product + b)
    assert bool(((product + b).abs() < 2.0 ** -4 * product.abs()).any())
    tol = (256 + h.blocks(width) + 2) * h.U * S + h.U * (S + b.abs())
    tol = tol + (want + tol) * h.HALF_STEP[torch.bfloat16]
    off = (got.double().cpu() - want).abs() - tol
    assert bool((off <= 0).all()), ((off > 0).sum().item(), off.max().item())
