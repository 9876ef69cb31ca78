"""The attention layer's operators at the edges of what their calls allow, on a host without a GPU."""
import ctypes

import pytest

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
