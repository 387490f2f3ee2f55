"""The cross entropy's kept plans are bounded, whatever the batches' row counts."""
import threading

import pytest


def _fake(monkeypatch):
    import recsys_linear_layers_amd as ll

    class Plan:
        made = 0

        def __init__(self, desc):
            Plan.made += 1
            self.rows = desc.N

    monkeypatch.setattr(ll, "XentPlan", Plan)  # a plan needs a device
    ll._xent_plans.clear()
    return ll, Plan


def test_plans_of_many_row_counts_do_not_pile_up(monkeypatch):
    torch = pytest.importorskip("torch")
    ll, Plan = _fake(monkeypatch)
    w = torch.zeros(50, 8).half()
    x = torch.zeros(3000, 8).half()
    try:
        for n in range(1, 2001):
            assert ll.xent_plan_for(x[:n], w).rows == n
            ll.xent_plan_for(x[:7], w)  # one in use all along
        assert Plan.made <= 2002 and 100 <= len(ll._xent_plans) <= 1000
        made = Plan.made
        for n in (7, 1999, 2000):
            assert ll.xent_plan_for(x[:n], w).rows == n
        assert Plan.made == made
        assert ll.xent_plan_for(x[:1], w).rows == 1 and Plan.made == made + 1
    finally:
        ll._xent_plans.clear()


def test_plans_asked_for_by_two_threads(monkeypatch):
    torch = pytest.importorskip("torch")
    ll, Plan = _fake(monkeypatch)
    w, x, wrong = torch.zeros(50, 8).half(), torch.zeros(3000, 8).half(), []

    def ask(k):
        try:
            wrong.extend(n for n in range(k, 1500, 2) for m in (n + 1, 3) if ll.xent_plan_for(x[:m], w).rows != m)
        except Exception as e:
            wrong.append(repr(e))

    threads = [threading.Thread(target=ask, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    ll._xent_plans.clear()
    assert not wrong
