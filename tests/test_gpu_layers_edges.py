"""Rotary positions and the distillation loss at the edges of what their calls allow, on the device.  Run on an MI355X:
pytest -m gpu."""
import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


@pytest.mark.parametrize("general", [False, True])
def test_arguments_of_as_many_values_in_other_rows(bd, general):
    """A teacher [K, N] for [N, K] and positions [L, B] for [B, L] are refused, by either way of making a call."""
    how = dict(stream=torch.cuda.current_stream()) if general else {}
    z = torch.randn(6, 40, device=DEV)
    index = torch.arange(18, dtype=torch.int32, device=DEV).reshape(6, 3)
    teacher, w = torch.randn(6, 3, device=DEV), torch.ones(6, device=DEV)
    loss, stat = bd.maxsim_distill_fwd(z, index, teacher, **how)
    bad = teacher.t().contiguous()
    with pytest.raises(ValueError, match="teacher"):
        bd.maxsim_distill_fwd(z, index, bad, **how)
    with pytest.raises(ValueError, match="teacher"):
        bd.maxsim_distill_bwd(w, z, stat, index, bad, **how)
    assert torch.equal(bd.maxsim_distill_fwd(z, index, teacher.flatten(), **how)[0], loss)
    x, f = torch.randn(2, 3, 4, 64, device=DEV), bd.rope_frequencies(64, device=DEV)[0]
    at = torch.randint(0, 1000, (2, 3), dtype=torch.int32, device=DEV)
    want = bd.maxsim_rope(x, f, positions=at, **how)
    assert torch.equal(bd.maxsim_rope(x, f, positions=at.flatten(), **how), want)
    with pytest.raises(ValueError, match="positions"):
        bd.maxsim_rope(x, f, positions=at.t().contiguous(), **how)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("N,V,K", [(511, 2048, 5), (511, 2049, 70), (512, 2049, 70), (512, 4096, 3), (512, 4097, 3)])
def test_rows_about_as_many_as_leave_a_wave_to_each(bd, N, V, K, dtype):
    g = torch.Generator().manual_seed(N + V)
    z, index = (3 * torch.randn(N, V, generator=g)).to(dtype), torch.randint(-1, V, (N, K), generator=g, dtype=torch.int32)
    teacher, dloss = 3 * torch.randn(N, K, generator=g), torch.rand(N, generator=g) + 0.5
    want = ref.distill(z, index, teacher, 0.8, dloss)
    d = [t.to(DEV) for t in (z, index, teacher, dloss)]
    loss, stat = bd.maxsim_distill_fwd(*d[:3], temperature=0.8)
    ref.check(loss, want["loss"], "loss")
    ref.check(bd.maxsim_distill_bwd(d[3], d[0], stat, *d[1:3], temperature=0.8), want["dscores"], "dscores")
