"""The attention layer's operators at the edges of what their calls allow, on a host without a GPU."""
import ctypes

import pytest
import torch

from late_interaction_retrieval_amd import binding as bd

A = 0x10000  # aligned non-null fake pointer: never dereferenced
BF16 = 1


def attn(**kw):
    a = bd._Attn()
    for n in ("q", "k", "v", "out"):
        setattr(a, n, bd._View(A, 4096, 128, 64))
    d = dict(B=2, max_q=5, max_k=9, Hq=2, Hk=2, D=64, dtype=BF16, left=-1, right=-1, sinks=0, zero_rest=0, scale=0.125, lse_step=1,
             rows_q=10, rows_k=18, cu_q=None, cu_k=None, q_lens=None, k_lens=None)
    d.update(kw)
    for n, v in d.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("max_k", [639, 640, 4096, 1 << 20])
def test_no_queries_are_not_split_over_keys(max_k, packed):
    """With max_q = 0 there is nothing to join, whatever rows of no sequence there are: no parts, and no workspace."""
    a = attn(max_q=0, max_k=max_k, cu_q=A if packed else None, rows_q=10)
    assert bd.lib().maxsim_attn_fwd_workspace_bytes(ctypes.byref(a)) == 0
    if max_k >= 4096:  # one query is split
        assert bd.lib().maxsim_attn_fwd_workspace_bytes(ctypes.byref(attn(max_q=1, max_k=max_k))) > 0


def test_rows_that_no_tile_can_be_loaded_from_are_copied():
    """attention() takes views of any layout: a contiguous one that starts off 16 bytes too."""
    flat = torch.zeros(2 * 3 * 4 * 64 + 8, dtype=torch.bfloat16)
    for at in (1, 4):
        t = flat[at:at + 2 * 3 * 4 * 64].view(2, 3, 4, 64)
        assert t.is_contiguous() and t.data_ptr() % 16 != 0
        u = bd._loadable(t)
        assert u.data_ptr() % 16 == 0 and u.is_contiguous() and torch.equal(u, t)
    whole = flat[:2 * 3 * 4 * 64].view(2, 3, 4, 64)
    assert bd._loadable(whole) is whole
    some = whole[:, :1, :, :36]  # rows of 72 bytes, 128 apart
    assert bd._loadable(some) is some
    for t in (whole.transpose(-1, -2), whole[:, :, :, 4:], whole[:, :, :, ::2]):
        u = bd._loadable(t)
        assert u.data_ptr() % 16 == 0 and u.is_contiguous() and torch.equal(u, t)
