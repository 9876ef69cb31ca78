"""Scales and codes of values held in e4m3 equal those of the plain fp32 form: a
scale is one product, max|v| times the fp32 value next to 1 / 448, a code the
nearest to v / scale.  Run on an MI355X: pytest -m gpu.

No tolerance: the plain form on the CPU makes the same two fp32 operations, each
rounded to nearest.  (The kernel's three-operation quotient can be a unit in the
last place off in about 1 of 10^7 cases; to move a code it would have to hit a
tie as well, about 1 in 1000 of these values: 10^-4 over all cases here.)"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INV = torch.tensor(np.float32(1) / np.float32(448))


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def plain(x, br):
    """Codes (as fp32) and scales of x [R, C], R and C multiples of 128."""
    R, C = x.shape
    cut = x.float().reshape(R // br, br, C // 128, 128)
    scale = cut.abs().amax(dim=(1, 3)) * INV
    codes = (cut / scale[:, None, :, None]).to(torch.float8_e4m3fn).float().reshape(R, C)
    return codes, scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("br", [1, 128])
def test_quantiser_equals_the_plain_form(bd, dtype, br):
    g = torch.Generator().manual_seed(11)
    x = torch.randn(512, 2048, generator=g) * torch.exp2(torch.randint(-20, 10, (512, 1), generator=g).float())
    x = x.to(dtype)
    q, s, qt, st = bd.maxsim_quant_fp8(x.to(DEV), block_rows=br, transposed=True)
    for got, got_s, want in ((q, s, plain(x, br)), (qt, st, plain(x.t().contiguous(), br))):
        assert torch.equal(got_s.cpu(), want[1])
        assert torch.equal(got.float().cpu(), want[0])


def test_norm_scales_are_products(bd):
    """A gain of 1 and rows of squares 1 on average: the norm changes no value, and its scales are the quantiser's."""
    x = torch.ones(64, 256)
    x[:, ::2] = -1
    y, s, _, r = bd.maxsim_rmsnorm_fwd(x.to(DEV), eps=0.0, out_dtype=torch.float8_e4m3fn, with_rstd=True)
    assert torch.all(r == 1) and torch.all(s.cpu() == INV)
    assert torch.equal(y.float().cpu(), x * 448)
