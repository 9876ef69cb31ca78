"""Attention at the edges of what its calls allow, forward and backward, on the device.  Run on an MI355X: pytest -m gpu."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def rand(*shape, dtype=BF16, seed=1):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("Lk", [5, 1000, 5000])
def test_no_queries_over_long_keys(bd, Lk, packed, general):
    """max_q = 0: rows of no sequence, if there are any, are zeros, and the keys get gradients of zeros."""
    how = dict(stream=torch.cuda.current_stream()) if general else {}
    k, v = rand(2, Lk, 2, 64, seed=2), rand(2, Lk, 2, 64, seed=3)
    if packed:
        q = rand(7, 4, 64)
        how.update(cu_q=torch.zeros(3, dtype=torch.int32, device=DEV), max_q=0)
    else:
        q = rand(2, 0, 4, 64)
    junk = torch.full((1 << 20,), 7.0, device=DEV)  # what an output made by the call may find in its memory
    del junk
    out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True, **how)
    assert out.shape == q.shape and torch.all(out == 0) and torch.all(lse == 0)
    dq, dk, dv = bd.maxsim_attn_bwd(torch.ones_like(q), q, k, v, out, lse, **how)
    for t, like in ((dq, q), (dk, k), (dv, v)):
        assert t.shape == like.shape and torch.all(t == 0)
