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


def meta(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_a_teacher_of_another_shape_is_refused():
    """As many values in other rows: [K, N] for [N, K]; a flat list of all rows' is taken."""
    raw = bd._distill_fwd.__wrapped__
    z, i = meta(4, 9, dtype=torch.float32), meta(4, 2, dtype=torch.int32)
    for bad in ((2, 4), (1, 8), (4, 2, 1)):
        with pytest.raises(ValueError, match="teacher"):
            raw(z, i, meta(*bad, dtype=torch.float32), 1.0, None, None, None)


def test_positions_of_another_shape_are_refused():
    """[L, B] for [B, L]; a flat list of all tokens' is taken."""
    raw, x, f = bd._rope.__wrapped__, meta(2, 3, 4, 64, dtype=torch.bfloat16), meta(32, dtype=torch.float64)
    for bad in ((3, 2), (1, 6), (2, 3, 1)):
        with pytest.raises(ValueError, match="positions"):
            raw(x, f, meta(*bad, dtype=torch.int32), None, "half", 1.0, False, None)
