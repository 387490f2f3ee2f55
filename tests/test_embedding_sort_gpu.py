"""The embedding gradient's sort at its own boundaries, with the tolerances of
test_embedding_gpu: one workgroup sorts up to 8192 tokens (8191, 8192: its last
step of 64 tokens per wave not quite and just full; 8193: the first radix sort),
digits of 10 bits, two, three and four passes, and scans over more than
eight workgroups' counts per wave (over 131072 tokens)."""
import pytest

from test_embedding_gpu import _gen, _grad_case, _ll

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,D,pad", [(8191, 700, 24, 0), (8192, 700, 24, 3), (8193, 700, 24, 0), (1024, 65537, 8, 0),
                                       (8192, 70000, 8, 0), (20000, 1000003, 8, 3), (20000, 1100000, 4, 0),
                                       (150000, 1000003, 4, 1), (150001, 1023, 8, 0), (300000, 1100000, 2, 0)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gradient_at_the_sorts_boundaries(dtype, T, V, D, pad, accumulate):
    """Ids from both ends of the table and some of everywhere, a few frequent, some without a gradient."""
    import torch
    g = _gen(T + V)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    u = torch.rand(T, generator=g, device="cuda")
    ids = torch.where(u < 0.2, V - 1 - ids % 5, torch.where(u < 0.3, ids % 3, ids))
    ids[torch.rand(T, generator=g, device="cuda") < 0.05] = V
    ids[torch.rand(T, generator=g, device="cuda") < 0.05] = 2 ** 33
    _grad_case(dtype, T, V, D, pad, ids, 0.75, 1, accumulate, g)


@pytest.mark.parametrize("V", [2 ** 30 + 5, 2 ** 31 - 2])
def test_gradient_into_a_table_of_more_than_2_to_30_rows(V):
    """Keys of 31 bits: four passes."""
    import torch
    ll = _ll()
    g = _gen(7)
    T = 9000
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[: T // 2] = V - 1 - ids[: T // 2] % 50
    dout = torch.ones((T, 1), dtype=torch.float16, device="cuda")
    got = ll.embedding_grad(ids, dout, V)
    rows, counts = torch.unique(ids, return_counts=True)
    assert torch.equal(got[rows, 0], counts.half())
    got[rows] = 0
    assert int(got.count_nonzero()) == 0
