"""The operators refuse tensors of a device that is not the current one: the
library would launch on the current one with the other's addresses.  (Stand-ins
for a second device; no GPU needed.)"""
import pytest


class Tensor:
    is_cuda = True

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


def test_tensors_of_another_device_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    import recsys_linear_layers_amd as ll
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    assert ll._stream_of(Tensor(1)) == 101
    with pytest.raises(ValueError, match="current device"):
        ll._stream_of(Tensor(0))


def test_no_plan_is_made_or_kept_for_tensors_of_another_device(monkeypatch):
    torch = pytest.importorskip("torch")
    import recsys_linear_layers_amd as ll
    monkeypatch.setattr(ll, "xent_plan_for", lambda *a: pytest.fail("a plan for the wrong device"))

    def refuse(t):
        raise ValueError("current device")

    monkeypatch.setattr(ll, "_stream_of", refuse)
    h = torch.zeros(5, 8).half()
    with pytest.raises(ValueError, match="current device"):
        ll.vocab_xent(h, h, torch.zeros(5, dtype=torch.int64))
