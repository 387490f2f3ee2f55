"""A next-item model trained with the library's operators from end to end.

Sequences of item ids (a user's history) predict, at every position, the id
that follows.  The model is what stands around a linear layer in a language
model or a sequential recommender:

    e  = scale * E[ids]                       embedding lookup
    n1 = layernorm(e);  h = relu(n1 W1^T + b1);  o = e + h W2^T
    n2 = layernorm(o);  loss = cross entropy of n2 E^T against the next ids

with the item table E used at both ends.  One step computes the loss and every
gradient with the operators' own gradient calls: ``vocab_xent_grad`` never holds
the [positions][items] logits, and ``embedding_grad(accumulate=True)`` adds the
lookup's gradient to the one the loss left in the same table.

    python examples/next_item.py [--steps 60]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import recsys_linear_layers_amd as ll  # noqa: E402

PAD = 0  # pads short histories; never predicted, and no gradient through the lookup


class NextItem:
    """Weights in bf16 beside fp32 master copies; gradients as the operators give them."""

    def __init__(self, items: int, width: int, hidden: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(shape, std):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.scale = math.sqrt(width)
        self.master = {
            "E": normal((items, width), 1 / math.sqrt(width)),
            "W1": normal((hidden, width), 1 / math.sqrt(width)),
            "W2": normal((width, hidden), 1 / math.sqrt(hidden)),
            "b1": torch.zeros(hidden, device="cuda"),
            "g1": torch.ones(width, device="cuda"), "c1": torch.zeros(width, device="cuda"),
            "g2": torch.ones(width, device="cuda"), "c2": torch.zeros(width, device="cuda"),
        }
        self.w = {}
        self.refresh()
        self.moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.master.items()}
        self.steps = 0

    def refresh(self):
        """bf16 matrices for the products; vectors stay fp32."""
        for k, v in self.master.items():
            self.w[k] = v.to(torch.bfloat16) if v.dim() == 2 else v

    def loss_and_grads(self, ids, target):
        """ids, target: int64 [positions] (target PAD: none).  Returns the mean loss
        and the gradients by name."""
        w, items = self.w, self.w["E"].shape[0]
        e = ll.embedding(w["E"], ids, scale=self.scale)
        n1, m1, r1 = ll.layernorm(e, w["g1"], w["c1"])
        h = ll.gemm(n1, w["W1"].t(), bias=w["b1"], act="relu")
        o = e + ll.gemm(h, w["W2"].t())
        n2, m2, r2 = ll.layernorm(o, w["g2"], w["c2"])
        live = target != PAD
        dloss = live.float() / live.sum().clamp_min(1)
        loss, _, dn2, dE = ll.vocab_xent_grad(n2, w["E"], target, dloss, ignore_index=PAD)

        do, dg2, dc2 = ll.layernorm_grad(dn2, o, m2, r2, w["g2"])
        dh = ll.gemm(do, w["W2"]) * (h > 0)
        dW2 = ll.gemm(do.t(), h, out_dtype=torch.float32)
        dW1 = ll.gemm(dh.t(), n1, out_dtype=torch.float32)
        dn1 = ll.gemm(dh, w["W1"])
        de, dg1, dc1 = ll.layernorm_grad(dn1, e, m1, r1, w["g1"])
        de += do
        ll.embedding_grad(ids, de, items, scale=self.scale, padding_idx=PAD, out=dE, accumulate=True)
        grads = {"E": dE, "W1": dW1, "W2": dW2, "b1": dh.float().sum(0), "g1": dg1, "c1": dc1, "g2": dg2, "c2": dc2}
        return (loss * dloss).sum(), grads

    def update(self, grads, lr: float = 2e-3, b1: float = 0.9, b2: float = 0.99):
        self.steps += 1
        for k, p in self.master.items():
            m, v = self.moments[k]
            d = grads[k].float()
            m.lerp_(d, 1 - b1)
            v.lerp_(d * d, 1 - b2)
            p.sub_(lr * (m / (1 - b1 ** self.steps)) / ((v / (1 - b2 ** self.steps)).sqrt() + 1e-8))
        self.refresh()


def histories(users: int, length: int, items: int, seed: int = 1):
    """Synthetic histories: each item is followed by a fixed successor most of the
    time; some histories are short and end in padding."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    successor = torch.randperm(items - 1, generator=g, device="cuda") + 1
    seq = torch.empty((users, length + 1), dtype=torch.int64, device="cuda")
    seq[:, 0] = torch.randint(1, items, (users,), generator=g, device="cuda")
    for t in range(length):
        other = torch.randint(1, items, (users,), generator=g, device="cuda")
        follow = torch.rand(users, generator=g, device="cuda") < 0.9
        seq[:, t + 1] = torch.where(follow, successor[seq[:, t] - 1], other)
    end = torch.randint(length // 2, length + 2, (users, 1), generator=g, device="cuda")
    seq[torch.arange(length + 1, device="cuda") >= end] = PAD
    return seq[:, :-1].reshape(-1), seq[:, 1:].reshape(-1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--items", type=int, default=5003)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--users", type=int, default=256)
    ap.add_argument("--length", type=int, default=32)
    a = ap.parse_args()
    model = NextItem(a.items, a.width, a.hidden)
    ids, target = histories(a.users, a.length, a.items)
    for step in range(a.steps):
        loss, grads = model.loss_and_grads(ids, target)
        model.update(grads)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {loss.item():.4f}", flush=True)
    # scoring: how likely the model finds each next item, from the loss alone
    e = ll.embedding(model.w["E"], ids[:1], scale=model.scale)
    n1, _, _ = ll.layernorm(e, model.w["g1"], model.w["c1"])
    o = e + ll.gemm(ll.gemm(n1, model.w["W1"].t(), bias=model.w["b1"], act="relu"), model.w["W2"].t())
    n2, _, _ = ll.layernorm(o, model.w["g2"], model.w["c2"])
    loss, _ = ll.vocab_xent(n2, model.w["E"], target[:1], ignore_index=PAD)
    print(f"log-likelihood of the first next item: {-loss.item():.4f}")


if __name__ == "__main__":
    main()
