"""The distillation loss and its gradient against their 64-bit form, on the device.  Run on an MI355X: pytest -m gpu."""
import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def make(N, V, K, dtype, seed=1, size=3.0):
    g = torch.Generator().manual_seed(seed)
    z = (size * torch.randn(N, V, generator=g)).to(dtype)
    index = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).to(torch.int32) if N and V >= K \
        else torch.zeros(N, K, dtype=torch.int32)
    return z, index.reshape(N, K), 3 * torch.randn(N, K, generator=g), torch.rand(N, generator=g) + 0.5


def check(bd, z, index, teacher, dloss, T=1.0, where=""):
    want = ref.distill(z, index, teacher, T, dloss)
    d = [t.to(DEV) for t in (z, index, teacher, dloss)]
    loss, stat = bd.maxsim_distill_fwd(*d[:3], temperature=T)
    ref.check(loss, want["loss"], where + " loss")
    got = bd.maxsim_distill_bwd(d[3], d[0], stat, d[1], d[2], temperature=T)
    assert got.dtype == z.dtype
    ref.check(got, want["dscores"], where + " dscores")
    again = d[0].clone()  # in place
    bd.maxsim_distill_bwd(d[3], again, stat, d[1], d[2], temperature=T, dscores=again)
    assert torch.equal(again, got)
    return loss, got


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=str)
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 7, 7), (64, 64, 16), (5, 1000, 100), (2, 1024, 3), (2, 1025, 64), (3, 4099, 130),
                                   (1, 8192, 1), (2, 20011, 1024), (70, 300, 0), (1, 70001, 33)])
@pytest.mark.parametrize("T", [1.0, 0.37])
def test_sizes(bd, dtype, N, V, K, T):
    check(bd, *make(N, V, K, dtype), T=T)


def test_rows_with_fewer_entries_none_and_the_same_one_twice(bd):
    z, index, teacher, dloss = make(6, 50, 5, F32)
    index[0, 3:] = -1                       # three entries
    index[1] = -1                           # none
    index[2] = torch.tensor([50, 1 << 30, -(1 << 31), 7, 8], dtype=torch.int32)  # out of range: two left
    index[3] = 11                           # one column five times
    index[4, 1] = index[4, 3]
    teacher[5] = -INF                       # entries that ask for nothing
    teacher[0, 1] = -INF
    loss, d = check(bd, z, index, teacher, dloss)
    assert loss[1] == 0 and torch.all(d[1] == 0) and loss[5] == 0 and torch.all(d[5] == 0)


@pytest.mark.parametrize("V", [40, 5000])
def test_columns_that_are_not_there(bd, V):
    """Scores of -infinity (candidates masked out) and of the type's lowest value."""
    z, index, teacher, dloss = make(4, V, 3, F32)
    for n in range(4):
        z[n, [c for c in range(V) if c not in index[n].tolist()][::2]] = -INF
    z[1, [c for c in range(V) if c not in index[1].tolist()]] = -INF  # only the teacher's
    z[2, index[2, 1].item()] = -INF                                  # one that the teacher asks for
    free = [c for c in range(V) if c not in index[3].tolist()]
    z[3, free] = torch.finfo(F32).min / 2
    loss, d = check(bd, z, index, teacher, dloss)
    assert loss[2] == INF and torch.isfinite(d).all()
    z[:] = -INF                                                      # no column at all
    dz = [t.to(DEV) for t in (z, index, teacher, dloss)]
    loss, stat = bd.maxsim_distill_fwd(*dz[:3])
    d = bd.maxsim_distill_bwd(dz[3], dz[0], stat, *dz[1:3])
    assert torch.all(loss == INF) and torch.isfinite(d).all() and abs(d.sum(1) + dz[3]).max() <= 1e-5


def test_large_scores_at_a_low_temperature(bd):
    """MaxSim's scores of 1024 query tokens at T = 0.02: exponents of tens of thousands."""
    z, index, teacher, dloss = make(8, 640, 16, F32, size=1.0)
    check(bd, 900 + z * 0.1, index, 900 + teacher * 0.05, dloss, T=0.02)


def test_nan_reaches_its_row_alone(bd):
    z, index, teacher, dloss = (t.to(DEV) for t in make(4, 100, 8, F32))
    z[1, 5] = float("nan")
    teacher[2] = float("nan")
    loss, stat = bd.maxsim_distill_fwd(z, index, teacher)
    d = bd.maxsim_distill_bwd(dloss, z, stat, index, teacher)
    assert torch.isnan(loss).tolist() == [False, True, True, False]
    assert torch.isnan(d).any(1).tolist() == [False, True, True, False]


def test_rows_of_a_wider_matrix(bd):
    z, index, teacher, dloss = make(5, 2000, 9, BF16)
    wide = torch.full((5, 2051), 9.0, dtype=BF16, device=DEV)
    wide[:, 3:2003] = z.to(DEV)
    kept = wide.clone()
    view = wide[:, 3:2003]
    i, t, g = index.to(DEV), teacher.to(DEV), dloss.to(DEV)
    loss, stat = bd.maxsim_distill_fwd(view, i, t)
    want = bd.maxsim_distill_fwd(z.to(DEV), i, t)
    assert torch.equal(loss, want[0]) and torch.equal(stat, want[1])
    d = bd.maxsim_distill_bwd(g, z.to(DEV), stat, i, t)
    bd.maxsim_distill_bwd(g, view, stat, i, t, dscores=view)
    assert torch.equal(view, d) and torch.equal(wide[:, :3], kept[:, :3]) and torch.equal(wide[:, 2003:], kept[:, 2003:])


def test_nothing_to_do(bd):
    e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    loss, stat = bd.maxsim_distill_fwd(e(0, 5), e(0, 2, dtype=torch.int32), e(0, 2))
    assert loss.shape == (0,)
    assert bd.maxsim_distill_bwd(e(0), e(0, 5), stat, e(0, 2, dtype=torch.int32), e(0, 2)).shape == (0, 5)
    loss, stat = bd.maxsim_distill_fwd(e(3, 0), torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.zeros(3, 2, device=DEV))
    assert torch.all(loss == 0)


def test_gradient_by_differences(bd):
    """Along a direction, fp32: (L(z + e d) - L(z - e d)) / 2 e in the 64-bit form, whose third derivative bounds its error."""
    z, index, teacher, dloss = make(3, 90, 6, F32)
    direction = torch.randn(3, 90, generator=torch.Generator().manual_seed(4)).double()
    _, d = check(bd, z, index, teacher, dloss)
    e = 1e-4
    value = lambda x: (ref.distill(x, index, teacher, 1.0)["loss"][0] * dloss.double()).sum()  # noqa: E731
    slope = (value(z.double() + e * direction) - value(z.double() - e * direction)) / (2 * e)
    # the softmax's third derivative along d is at most 6 max|d|^3 a row; the gradient is within its own bound
    bound = (dloss.double() * e * e * direction.abs().amax(1) ** 3).sum() + 1e-9 + \
        (ref.distill(z, index, teacher, 1.0, dloss)["dscores"][1] * direction.abs()).sum()
    assert abs(slope - (d.double().cpu() * direction).sum()) <= bound


def test_autograd_of_scores(bd):
    z, index, teacher, dloss = (t.to(DEV) for t in make(7, 33, 4, F32))
    z.requires_grad_()
    loss = bd.distill_loss(z, index, teacher, temperature=2.0)
    got, = torch.autograd.grad((loss * dloss).sum(), z)
    _, stat = bd.maxsim_distill_fwd(z.detach(), index, teacher, temperature=2.0)
    assert torch.equal(got, bd.maxsim_distill_bwd(dloss, z.detach(), stat, index, teacher, temperature=2.0))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_scores_past_the_last_cache(bd, dtype):
    """Over 256 MB, whose loads and stores go past the caches: the same values as its rows by themselves."""
    N, V = 70, (1 << 20) * (2 if dtype == BF16 else 1) + 3
    g = torch.Generator(device=DEV).manual_seed(3)
    z = (3 * torch.randn(N, V, device=DEV, generator=g)).to(dtype)
    index = torch.randint(0, V, (N, 9), device=DEV, generator=g, dtype=torch.int32)
    index[5, 3] = index[5, 7]
    teacher, dloss = torch.randn(N, 9, device=DEV, generator=g), torch.rand(N, device=DEV, generator=g)
    loss, stat = bd.maxsim_distill_fwd(z, index, teacher)
    d = bd.maxsim_distill_bwd(dloss, z, stat, index, teacher)
    for a in range(0, N, 10):
        r = slice(a, a + 10)
        part = bd.maxsim_distill_bwd(dloss[r].contiguous(), z[r], stat[r].contiguous(), index[r].contiguous(), teacher[r].contiguous())
        assert torch.equal(part, d[r])
    want = ref.distill(z[5:6].cpu(), index[5:6].cpu(), teacher[5:6].cpu(), 1.0, dloss[5:6].cpu())
    ref.check(loss[5:6], want["loss"], "loss")
    ref.check(d[5:6], want["dscores"], "dscores")
    bd.maxsim_distill_bwd(dloss, z, stat, index, teacher, dscores=z)
    assert torch.equal(z, d)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("V,K", [(4095, 70), (4096, 33), (4097, 300)])
def test_rows_about_as_long_as_a_wave_takes_by_itself(bd, dtype, V, K):
    z, index, teacher, dloss = make(9, V, K, dtype, seed=20)
    index[3, ::3] = -2
    index[4, 1:] = V + 2
    check(bd, z, index, teacher, dloss, T=0.7)
