"""Rotary positions against their 64-bit form, on the device.  Run on an MI355X: pytest -m gpu."""
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


def check(bd, x, rotary, layout, dtype, positions=None, offsets=None, inverse=False, scale=1.0, stretch=1.0, **kw):
    """x: [B, L, H, D] or [T, H, D] on the device."""
    f, more = bd.rope_frequencies(rotary, stretch=stretch, device=DEV)
    y = bd.maxsim_rope(x, f, positions=positions, offsets=offsets, layout=layout, scale=scale * more, inverse=inverse, **kw)
    B, L = (x.shape[0], x.shape[1]) if x.dim() == 4 else (1, x.shape[0])
    if positions is not None:
        at = positions.reshape(-1)
    else:
        at = torch.arange(L, device=DEV).repeat(B)
        if offsets is not None:
            at = at + offsets.long().repeat_interleave(L)
    want = ref.rope(x.detach().cpu().reshape((-1,) + x.shape[-2:]), f.cpu(), at.cpu(), layout, scale * more, inverse)
    assert y.shape == x.shape and y.dtype == dtype
    ref.check(y, want, "%s %s %s" % (tuple(x.shape), rotary, layout))
    return y


def rand(*shape, dtype=F32, seed=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=str)
@pytest.mark.parametrize("shape,rotary", [((1, 1, 1, 2), 2), ((2, 3, 5, 7), 6), ((1, 17, 3, 64), 64), ((3, 9, 2, 128), 64),
                                          ((1, 5, 7, 80), 48), ((2, 33, 4, 128), 128), ((1, 3, 2, 1024), 1022),
                                          ((4, 1, 20, 64), 34), ((1, 300, 1, 66), 66)], ids=str)
def test_sizes(bd, layout, dtype, shape, rotary):
    check(bd, rand(*shape, dtype=dtype), rotary, layout, dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_and_stretched_frequencies(bd, layout):
    at = torch.tensor([0, 1, -5, 4095, 131071, 1 << 20, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device=DEV)
    check(bd, rand(8, 3, 128), 128, layout, F32, positions=at, stretch=8.0)


@pytest.mark.parametrize("inverse", [False, True])
def test_offsets_given_positions_and_the_inverse(bd, inverse):
    x = rand(5, 4, 6, 64, dtype=BF16)
    offsets = torch.tensor([0, 7, 100000, -3, 12], dtype=torch.int32, device=DEV)
    a = check(bd, x, 64, "half", BF16, offsets=offsets, inverse=inverse)
    at = (offsets[:, None] + torch.arange(4, device=DEV, dtype=torch.int32)).contiguous()
    b = check(bd, x, 64, "half", BF16, positions=at, inverse=inverse)
    assert torch.equal(a, b)


def test_heads_of_a_wider_projection_in_place_and_elsewhere(bd):
    """The first 10 of 14 heads' rows, in place; what lies beside them stays.  Then to an output of another layout."""
    wide = rand(3, 21, 14, 40, dtype=F16)
    kept = wide.clone()
    x = wide[:, :, :10]
    want = check(bd, x.clone(), 24, "interleaved", F16)
    elsewhere = torch.full((3, 10, 21, 40), 7.0, dtype=F16, device=DEV)
    f, scale = bd.rope_frequencies(24, device=DEV)
    got = bd.maxsim_rope(x, f, layout="interleaved", scale=scale, out=elsewhere.transpose(1, 2))
    assert torch.equal(got, want) and torch.equal(wide, kept)
    bd.maxsim_rope(x, f, layout="interleaved", scale=scale, out=x)
    assert torch.equal(x, want) and torch.equal(wide[:, :, 10:], kept[:, :, 10:])


def test_rows_of_any_alignment(bd):
    flat = rand(1 + 2 * 5 * 3 * 66, dtype=F16)
    x = flat[1:].reshape(2, 5, 3, 66)
    check(bd, x, 66, "half", F16)
    check(bd, x[..., 1:], 64, "interleaved", F16)


def test_nothing_to_do(bd):
    f, _ = bd.rope_frequencies(8, device=DEV)
    for shape in ((0, 4, 2, 8), (3, 0, 2, 8), (0, 2, 8)):
        assert bd.maxsim_rope(torch.empty(shape, device=DEV), f).shape == shape


def test_not_finite_values_stay_in_their_pairs(bd):
    x = rand(1, 6, 2, 16)
    x[0, 2, 1, 3] = float("nan")
    x[0, 4, 0, 9] = float("inf")
    f, _ = bd.rope_frequencies(16, device=DEV)
    y = bd.maxsim_rope(x, f)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 2, 1, 3] = want[0, 2, 1, 11] = want[0, 4, 0, 9] = want[0, 4, 0, 1] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(bd, layout):
    """Against the formula's: the transpose of a rotation is its inverse; and <R x, y> = <x, R' y>."""
    x = rand(2, 9, 3, 20).requires_grad_()
    g = rand(2, 9, 3, 20, seed=2)
    f, scale = bd.rope_frequencies(12, stretch=4.0, device=DEV)
    offsets = torch.tensor([3, 50], dtype=torch.int32, device=DEV)
    y = bd.rope(x, f, offsets=offsets, layout=layout, scale=scale)
    dx, = torch.autograd.grad(y, x, g)
    at = (offsets.long()[:, None] + torch.arange(9, device=DEV)).reshape(-1).cpu()
    ref.check(dx, ref.rope(g.cpu().reshape(-1, 3, 20), f.cpu(), at, layout, scale, inverse=True), "dx")
    left, right = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    size = (y.double() * g.double()).abs().sum()
    assert abs(left - right) <= 32 * ref.U * size  # each value within 16 u of its own size
    # by differences, of a linear map: exact but for roundings
    d = rand(2, 9, 3, 20, seed=3)
    with torch.no_grad():
        moved = bd.rope(x + d, f, offsets=offsets, layout=layout, scale=scale)
    change = ((moved - y).double() * g.double()).sum()
    size = ((moved.abs() + y.abs()).double() * g.double().abs()).sum()
    assert abs(change - (d.double() * dx.double()).sum()) <= 32 * ref.U * size


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rows_past_the_last_cache(bd, layout):
    """Over 256 MB in and out, whose loads go past the caches: the same values as some of its rows by themselves."""
    x = torch.randn(3, 12000, 20, 100, device=DEV, dtype=torch.float32).to(BF16)
    f, _ = bd.rope_frequencies(66, device=DEV)
    y = bd.maxsim_rope(x, f, layout=layout)
    assert torch.equal(y[1, :500], bd.maxsim_rope(x[1, :500], f, layout=layout))
    assert torch.equal(y[2, :700], bd.maxsim_rope(x[2, :700], f, layout=layout))
    want = y.clone()
    bd.maxsim_rope(x, f, layout=layout, out=x)
    assert torch.equal(x, want)
