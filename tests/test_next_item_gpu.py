"""The operators together: examples/next_item.py's gradients against torch's
automatic differentiation of the same model in 64 bits, and its training loss."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("next_item", os.path.join(ROOT, "examples", "next_item.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(model, ids, target, pad):
    """Loss and gradients on the host, in 64 bits, from the same bf16 weights."""
    import torch
    F = torch.nn.functional
    w = {k: v.detach().double().cpu().requires_grad_() for k, v in model.w.items()}
    ids, target = ids.cpu(), target.cpu()
    D = w["E"].shape[1]
    table = w["E"]
    e = table[ids]
    e = torch.where((ids == pad)[:, None], e.detach(), e) * model.scale  # no gradient through padding
    n1 = F.layer_norm(e, (D,), w["g1"], w["c1"], 1e-5)
    h = torch.relu(n1 @ w["W1"].T + w["b1"])
    o = e + h @ w["W2"].T
    n2 = F.layer_norm(o, (D,), w["g2"], w["c2"], 1e-5)
    loss = F.cross_entropy(n2 @ table.T, target, ignore_index=pad)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in w.items()}


@pytest.mark.parametrize("items,width,hidden,users,length", [(301, 64, 96, 9, 12), (2003, 200, 264, 70, 11)])
def test_gradients_of_the_whole_model(items, width, hidden, users, length):
    """The 64-bit model keeps every activation exact; here each of the ~10
    tensors along a gradient's way is rounded to bf16 once (2^-9 of its size on
    average, 2^-8 at most) and may flip a relu near 0, so the gradients agree to
    a few hundredths of their norm."""
    import torch
    ex = _example()
    model = ex.NextItem(items, width, hidden, seed=3)
    ids, target = ex.histories(users, length, items, seed=4)
    assert bool((target == ex.PAD).any())
    loss, grads = model.loss_and_grads(ids, target)
    ref_loss, ref = _reference(model, ids, target, ex.PAD)
    assert abs(loss.item() - ref_loss) <= 0.02 * ref_loss
    for k, g in grads.items():
        err = (g.double().cpu() - ref[k]).norm() / ref[k].norm()
        assert err <= 0.05, (k, err.item())
    assert all(bool(torch.isfinite(g).all()) for g in grads.values())


def test_training_learns_the_successors():
    ex = _example()
    model = ex.NextItem(501, 128, 256, seed=1)
    ids, target = ex.histories(128, 24, 501, seed=2)
    first = None
    for _ in range(60):
        loss, grads = model.loss_and_grads(ids, target)
        first = first if first is not None else loss.item()
        model.update(grads)
    # from about the log of the items (plus the logits' spread) to well under half
    assert first > 0.9 * math.log(501) and loss.item() < 0.5 * first, (first, loss.item())
