"""The embedding operators at the largest sizes their entries take: the bounds
on the host, and on the GPU widths and token counts whose indexes come near 32
bits.  Values are whole numbers that every step holds exactly."""
import ctypes

import pytest

from test_operator_refusals import P, Q, R, _embed, _embed_grad, _status

MOST = 2 ** 31 - 2 ** 12  # tokens, columns


def _ll():
    import recsys_linear_layers_amd as ll
    return ll


@pytest.mark.parametrize("size", ["T", "D"])
def test_sizes_past_32_bit_indexes_are_refused(size):
    """Indexes are rounded up to whole workgroups and steps: the last 4096 sizes below 2^31 have no room for that."""
    ll = _ll()
    n = ctypes.c_size_t()
    for over in (MOST + 1, 2 ** 31 - 2):
        kw = dict(T=over) if size == "T" else dict(D=over, stride_table=over, stride_out=over)
        assert _status(ll._lib.embed_run, _embed(**kw), P, Q, R, None) == "LL_ERR_UNSUPPORTED"
        kw = dict(T=over) if size == "T" else dict(D=over, stride_dout=over, stride_dtable=over)
        assert _status(ll._lib.embed_grad_workspace_size, _embed_grad(**kw), ctypes.byref(n)) == "LL_ERR_UNSUPPORTED"
        assert _status(ll._lib.embed_grad_run, _embed_grad(**kw), P, Q, R, None, 0, None) == "LL_ERR_UNSUPPORTED"
    kw = dict(T=MOST) if size == "T" else dict(D=MOST, stride_dout=MOST, stride_dtable=MOST)
    assert _status(ll._lib.embed_grad_workspace_size, _embed_grad(**kw), ctypes.byref(n)) == "LL_OK"


@pytest.mark.gpu
def test_lookup_of_the_widest_row():
    import torch
    ll = _ll()
    table = torch.full((1, MOST), 3.0, dtype=torch.bfloat16, device="cuda")
    table[0, -1] = 5.0
    out = ll.embedding(table, torch.zeros(1, dtype=torch.int64, device="cuda"), scale=2.0)
    assert float(out[0, -1]) == 10.0 and bool((out[0, :-1] == 6.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T", [3, 17])
def test_gradient_of_rows_wider_than_2_to_30(T, accumulate):
    """Steps over the columns pass 2^31 behind the last one; 17 tokens of a row hold a whole chunk."""
    import torch
    ll = _ll()
    D = 2 ** 30 + 3 * 512 + 8
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")
    dout = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    for t in range(T):
        dout[t] = t + 1
    dout[:, -1] = 1
    out = torch.full((1, D), 1.0, dtype=torch.bfloat16, device="cuda")
    ll.embedding_grad(ids, dout, 1, out=out, accumulate=accumulate)
    want = T * (T + 1) // 2 + accumulate
    assert bool((out[0, :-1] == want).all()) and float(out[0, -1]) == T + accumulate


@pytest.mark.gpu
def test_gradient_in_more_workgroups_than_one_launch_takes():
    """2^25 tokens of two blocks of columns: more than 2^32 threads."""
    import torch
    ll = _ll()
    T, V, D = 2 ** 25 + 1000, 2 ** 20, 513
    ids = torch.arange(T, device="cuda") % V
    dout = torch.ones((T, D), dtype=torch.bfloat16, device="cuda")
    got = ll.embedding_grad(ids, dout, V)
    counts = torch.bincount(ids, minlength=V).to(torch.bfloat16)
    assert bool((got == counts[:, None]).all())
