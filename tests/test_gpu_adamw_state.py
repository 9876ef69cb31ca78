"""The optimiser's state over several steps beside the plain fp32 form, each from its own state: the moments are made of
the same elementary fp32 operations, so they stay equal, and with them the 8-bit codes and scales.
Run on an MI355X: pytest -m gpu.

No tolerance: m is beta1 m rounded and a multiply-add, v beta2 v and g g rounded and a multiply-add; a scale is one
product, a code the nearest to a quotient.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B1, B2 = 0.9, 0.999
INV = float(np.float32(1) / np.float32(448))


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def f32(x):
    return float(np.float32(x))


def fma(a, scalar, b):
    """a * scalar + b with one rounding to fp32.  The product is exact in 64 bits; the sum is rounded to odd there (a
    sum that is not exact gets an odd last bit), which the rounding to 32 bits cannot mistake for a tie."""
    p, b = a.double() * f32(scalar), b.double()
    s = p + b
    back = s - p
    err = (p - (s - back)) + (b - back)     # what the sum lost, exactly
    away = torch.where(err > 0, torch.inf, -torch.inf).double()
    even = (s.view(torch.int64) & 1) == 0
    return torch.where((err != 0) & even, torch.nextafter(s, away), s).float()


def moments(m, v, g):
    return fma(g, 1 - B1, m * f32(B1)), fma(g * g, 1 - B2, v * f32(B2))


def pack(x, root=False):
    """Codes as fp32 and scales of x [n], n a multiple of 128; a root that is not 0 is never held as 0."""
    cut = x.reshape(-1, 128)
    top = cut.abs().amax(1)
    scale = torch.where(top < 2.0 ** -100, torch.ones_like(top), top * INV)
    t = cut / scale[:, None]
    if root:
        t = torch.where(t > 0, t.clamp_min(2.0 ** -9), t)
    return t.clamp(-448, 448).to(torch.float8_e4m3fn).float(), scale


def gradient(n, t, dtype):
    g = torch.Generator(DEV).manual_seed(100 + t)
    return (torch.randn(n, device=DEV, generator=g) * 1e-3).to(dtype)


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16], ids=str)
def test_8_bit_states_stay_with_the_plain_form(bd, grad):
    n = 1 << 23
    tab = bd.AdamWTensors.zeros([torch.zeros(n, device=DEV)], torch.float8_e4m3fn)
    m = v = torch.zeros(n, device=DEV)
    for t in range(1, 6):
        g = gradient(n, t, grad)
        bd.maxsim_adamw(tab, [g], t, 1e-3, B1, B2)
        m, v = moments(m, v, g.float())
        (qm, sm), (qv, sv) = pack(m), pack(v.sqrt(), True)
        assert torch.equal(tab.m_scales[0], sm) and torch.equal(tab.v_scales[0], sv), t
        assert torch.equal(tab.m[0].float(), qm.flatten()) and torch.equal(tab.v[0].float(), qv.flatten()), t
        m, v = (qm * sm[:, None]).flatten(), (qv * sv[:, None]).square().flatten()


def test_fp32_states_stay_with_the_plain_form(bd):
    n = 1 << 22
    tab = bd.AdamWTensors.zeros([torch.zeros(n, device=DEV)])
    m = v = torch.zeros(n, device=DEV)
    for t in range(1, 5):
        g = gradient(n, t, torch.float32)
        bd.maxsim_adamw(tab, [g], t, 1e-3, B1, B2)
        m, v = moments(m, v, g)
        assert torch.equal(tab.m[0], m) and torch.equal(tab.v[0], v), t


@pytest.mark.parametrize("largest", [1.0, 1e-9, 1.85e-16, 1e-18])
def test_a_second_moment_is_never_lost(bd, largest):
    """Blocks whose roots reach down to where their squares leave fp32: with eps = 0 a moment read as 0 would be a division
    by 0.  1.85e-16: the largest root is 5.85e-18, the smallest code's value 2.55e-23 and its square 6.5e-46, less than
    half of the smallest fp32 value.  The second step's m / sqrt(v) is at most 1.8 times (codes of m and of the root off by
    half a step each at the smallest, 1.5 and 2 / 3 of them) the first step's, 1: 8 is safe."""
    small = 1.18e-21   # its square times 1 - beta2 rounds to the smallest fp32 value
    g = torch.full((256,), small, device=DEV)
    g[5] = largest
    g[200] = 0.0
    tab = bd.AdamWTensors.zeros([torch.zeros(256, device=DEV)], torch.float8_e4m3fn)
    bd.maxsim_adamw(tab, [g], 1, 2.0 ** -10, B1, B2, 0.0, 0.0)
    # g[200] gives 0 / 0, as the formula has it; all others move
    ok = torch.arange(256, device=DEV) != 200
    first = tab.params[0].clone()
    assert torch.isnan(first[200]) and torch.isfinite(first[ok]).all() and torch.all(tab.v[0].float()[ok] > 0)
    bd.maxsim_adamw(tab, [torch.zeros_like(g)], 2, 2.0 ** -10, B1, B2, 0.0, 0.0)
    assert torch.all((tab.params[0] - first)[ok].abs() <= 8 * 2.0 ** -10)
