"""The order in which the norms' gradients add up rows is one of the sizes alone: the
sums bit for bit as 512 partial rows give them, joined as 16 runs of 32, on any device.

Rows and their gradients are bf16 and the rows' scale is a power of two, so that a
product has 16 bits; beside an fp32 sum it fits 53, so 64 bits rounded once are fma."""
import pytest

pytestmark = pytest.mark.gpu
PARTIALS = 512


def _inputs(N, D):
    import torch
    import helpers8 as h
    dy, x = (h.normal((N, D), seed, torch.bfloat16) for seed in (1, 2))
    rstd = 2.0 ** torch.randint(-2, 3, (N,), generator=torch.Generator().manual_seed(3)).float()
    return dy, x, rstd


def _partials(term, per_step, product):
    """[blocks][D] sums of term [N][D] (64 bits): workgroup b takes rows b, b + blocks, ...
    of per_step rows each, a running fp32 sum for each of them, added up in order."""
    import torch
    N, D = term.shape
    steps = -(-N // per_step)
    blocks = max(1, min(steps, PARTIALS))
    turns = -(-steps // blocks)
    t = torch.nn.functional.pad(term, (0, 0, 0, turns * blocks * per_step - N)).view(turns, blocks, per_step, D)
    acc = torch.zeros(blocks, per_step, D)
    for k in range(turns):
        acc = (acc.double() + t[k]).float() if product else acc + t[k].float()
    out = acc[:, 0]
    for y in range(1, per_step):
        out = out + acc[:, y]
    return out


def _joined(partial):
    """Sixteen runs, each from zero, added up in order."""
    import torch
    n = len(partial)
    out = None
    for w in range(16):
        s = torch.zeros(partial.shape[1])
        for k in range(n * w // 16, n * (w + 1) // 16):
            s = s + partial[k]
        out = s if out is None else out + s
    return out


# columns, rows that a workgroup takes at a time: four of up to 512 columns (one wave each), else one
SIZES = [(40, 7001, 4), (500, 2600, 4), (40, 2049, 4), (5000, 1300, 1), (16400, 1101, 1)]


@pytest.mark.parametrize("D,N,per_step", SIZES)
def test_rmsnorm(D, N, per_step):
    import torch
    import recsys_linear_layers_amd as ll
    dy, h, rstd = _inputs(N, D)
    gamma = torch.ones(D, device="cuda")
    _, got = ll.rmsnorm_grad(dy.cuda(), h.cuda(), rstd.cuda(), gamma)
    term = dy.double() * (h.double() * rstd.double()[:, None])
    assert torch.equal(got.cpu(), _joined(_partials(term, per_step, True)))


@pytest.mark.parametrize("D,N,per_step", SIZES)
def test_layernorm(D, N, per_step):
    import torch
    import recsys_linear_layers_amd as ll
    dy, x, rstd = _inputs(N, D)
    mean, gamma = torch.zeros(N, device="cuda"), torch.ones(D, device="cuda")  # with a mean of 0 x * rstd is exact
    _, dgamma, dbeta = ll.layernorm_grad(dy.cuda(), x.cuda(), mean, rstd.cuda(), gamma)
    term = dy.double() * (x.double() * rstd.double()[:, None])
    assert torch.equal(dgamma.cpu(), _joined(_partials(term, per_step, True)))
    assert torch.equal(dbeta.cpu(), _joined(_partials(dy.double(), per_step, False)))
