"""RMS norm, with the residual and the 8-bit outputs, and its backward against
the 64-bit forms of encoder_ref.  Run on an MI355X: pytest -m gpu.

Tolerances: the kernel adds a row's squares in fp32, at most 64 in one lane and
then over lanes and waves, so r is off by at most 2^-18 relative; the two
products after it and the rounding to the output's type come on top."""
import numpy as np
import pytest
import torch

import encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ERR = 2.0 ** -18 + 4 * ref.U
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def rows(seed, R, H, dtype, scale=1.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.standard_normal((R, H)) * scale).to(dtype)


def check(got, want, dtype, err, where, floor=0.0):
    got = got.double().cpu()
    tol = want.abs() * (ref.half_step(dtype) * (1 + 1e-3) + err) + floor
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = (got - want).abs() > tol
    assert not bad.any(), "%s: %d off, worst %.3g" % (where, int(bad.sum()), float(((got - want).abs() / tol).max()))


# one value, an odd few, each plan of threads to a row with its first and last width, odd tails
SHAPES = [(1, 1), (3, 7), (17, 128), (5, 129), (33, 512), (4, 513), (7, 769), (9, 1024), (2, 1025), (5, 2048), (3, 2049),
          (2, 4097), (3, 8192), (2, 8193), (2, 16385), (1, 32768), (1000, 128), (300, 100)]


@pytest.mark.parametrize("R,H", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_forward(bd, R, H, dtype):
    x, w = rows(R + H, R, H, dtype), 1 + 0.1 * rows(1, 1, H, torch.float32)[0]
    res = rows(R + H + 1, R, H, dtype, 2.0)
    for weight, residual in ((None, None), (w.to(dtype), res), (w, res)):
        h, r, y = ref.rmsnorm(x, weight, residual, 1e-6)
        to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        for out in (None, torch.int8, torch.float8_e4m3fn, torch.float32):
            got, scale, total, rstd = bd.maxsim_rmsnorm_fwd(to(x), to(weight), 1e-6, residual=to(residual),
                                                            out_dtype=out, with_rstd=True)
            where = "%s %s" % (out, None if weight is None else weight.dtype)
            check(rstd, r, torch.float32, ERR, where + " rstd")
            if residual is None:
                assert total is None
            else:  # the sum is exact in fp32 for 16-bit rows, and rounded once
                check(total, h, dtype, 2 * ref.U if dtype == torch.float32 else ref.U, where + " sum")
            err = ERR
            if residual is not None:  # where x + residual cancels in fp32, y is off by that rounding
                err = ERR
            floor = float(y.abs().max()) * 2 * ref.U
            if out == torch.int8:
                assert scale.shape == (R,)
                ref.check_held(got, scale[:, None], y, 1, H, "i8", err, where)
            elif out == torch.float8_e4m3fn:
                assert scale.shape == (R, -(-H // 128))
                ref.check_held(got, scale, y, 1, 128, "e4m3", err, where)
            else:
                assert scale is None
                check(got, y, out or dtype, err, where, floor)


@pytest.mark.parametrize("R,H", [(1, 1), (3, 7), (40, 128), (37, 129), (19, 769), (9, 1024), (2500, 128), (1500, 513),
                                 (1100, 2048), (6, 4099), (3, 8192), (2, 20000)])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_backward(bd, R, H, dtype):
    dy, h = rows(R * H, R, H, dtype), rows(R * H + 1, R, H, dtype)
    ds = rows(R * H + 2, R, H, dtype, 0.3)
    w = 1 + 0.1 * rows(2, 1, H, torch.float32)[0]
    _, r, _ = ref.rmsnorm(h, None, None, 1e-6)
    r = r.float()
    for weight, dsum in ((None, None), (w.to(dtype), ds), (w, None)):
        dx, dw, dx_size, dw_size = ref.rmsnorm_bwd(dy, h, r, weight, dsum)
        to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        got, gw = bd.maxsim_rmsnorm_bwd(to(dy), to(h), to(r), to(weight), dsum=to(dsum))
        tol = ref.half_step(dtype) * dx.abs() * (1 + 1e-3) + 2.0 ** -18 * dx_size
        if dtype == torch.float16:
            tol = tol + 2.0 ** -25
        assert torch.all((got.double().cpu() - dx).abs() <= tol)
        # a column's terms: at most 64 in a thread, 16 rows of a workgroup, 64 partial sums, 16 runs
        assert torch.all((gw.double().cpu() - dw).abs() <= 2.0 ** -16 * dw_size)
        again = bd.maxsim_rmsnorm_bwd(to(dy), to(h), to(r), to(weight), dsum=to(dsum))
        assert torch.equal(again[0], got) and torch.equal(again[1], gw)
        assert bd.maxsim_rmsnorm_bwd(to(dy), to(h), to(r), to(weight), dsum=to(dsum), with_dweight=False)[1] is None


def test_gradient_against_differences(bd):
    """The kernel's gradient of <dy, y> + <ds, sum> by central differences of the 64-bit forward."""
    R, H = 3, 40
    x, res = rows(1, R, H, torch.float32), rows(2, R, H, torch.float32)
    w, dy, ds = rows(3, 1, H, torch.float32)[0], rows(4, R, H, torch.float32), rows(5, R, H, torch.float32)

    def loss(xx, ww):
        h, _, y = ref.rmsnorm(xx, ww, res, 1e-6)
        return float((y * dy.double()).sum() + (h * ds.double()).sum())

    h, r, _ = ref.rmsnorm(x, w, res, 1e-6)
    dx, dw = bd.maxsim_rmsnorm_bwd(dy.to(DEV), h.float().to(DEV), r.float().to(DEV), w.to(DEV), dsum=ds.to(DEV))
    step = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros(R, H, dtype=torch.float64)
        e[i, j] = step
        diff = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * step)
        assert abs(diff - float(dx[i, j])) <= 1e-4 * max(1, abs(diff))
        diff = (loss(x.double(), w.double() + e[i]) - loss(x.double(), w.double() - e[i])) / (2 * step)
        assert abs(diff - float(dw[j])) <= 1e-4 * max(1, abs(diff))


@pytest.mark.parametrize("off,pitch", [(0, 200), (1, 201), (3, 208)])
def test_pitches_and_alignments(bd, off, pitch):
    """Slices of wider rows at any element; nothing outside the rows is written."""
    R, H, dt = 9, 150, torch.bfloat16
    wide = rows(5, R, pitch + off, dt).to(DEV)
    x = wide[:, off:off + H]
    _, _, y = ref.rmsnorm(x.cpu(), None, None, 1e-6)
    for out in (dt, torch.int8, torch.float8_e4m3fn):
        buf = torch.full((R + 2, pitch + off), 7, dtype=torch.float32, device=DEV).to(out)
        into = buf[1:-1, off:off + H]
        got, scale, _, _ = bd.maxsim_rmsnorm_fwd(x, out_dtype=out, y=into)
        assert got.data_ptr() == into.data_ptr()
        if out == dt:
            check(into, y, dt, ERR, "pitch")
        else:
            kind = "i8" if out == torch.int8 else "e4m3"
            s = scale[:, None] if out == torch.int8 else scale
            ref.check_held(into, s, y, 1, H if out == torch.int8 else 128, kind, ERR, "pitch")
        rest = buf.float()
        rest[1:-1, off:off + H] = 7
        assert torch.all(rest == 7), "a value outside the rows was written"
    h3 = torch.zeros(2, 3, H, dtype=dt, device=DEV)
    assert bd.maxsim_rmsnorm_fwd(h3, out_dtype=torch.float8_e4m3fn)[1].shape == (2, 3, 2)


def test_in_place(bd):
    """sum over residual, y over x, dx over dy: the same results as with memory of their own."""
    R, H = 50, 700
    x, res = rows(1, R, H, torch.bfloat16).to(DEV), rows(2, R, H, torch.bfloat16).to(DEV)
    y, _, h, r = bd.maxsim_rmsnorm_fwd(x, residual=res, with_rstd=True)
    x2, res2 = x.clone(), res.clone()
    bd.maxsim_rmsnorm_fwd(x2, residual=res2, y=x2, sum=res2)
    assert torch.equal(x2, y) and torch.equal(res2, h)
    # few rows (one launch, or two in place) and many
    for R, H in ((50, 700), (1000, 1000), (512, 8000), (3000, 300)):
        h, dy = rows(2, R, H, torch.bfloat16).to(DEV), rows(3, R, H, torch.bfloat16).to(DEV)
        ds = rows(4, R, H, torch.bfloat16).to(DEV)
        _, _, _, r = bd.maxsim_rmsnorm_fwd(h, with_rstd=True)
        dx, dw = bd.maxsim_rmsnorm_bwd(dy, h, r, dsum=ds)
        for over in range(3):
            ins = [dy.clone(), h.clone(), ds.clone()]
            dx2, dw2 = bd.maxsim_rmsnorm_bwd(ins[0], ins[1], r, dsum=ins[2], dx=ins[over])
            assert dx2 is ins[over] and torch.equal(dx2, dx) and torch.equal(dw2, dw), (R, H, over)


def test_zero_rows_and_extremes(bd):
    H = 256
    x = torch.zeros(6, H)
    x[1] = 1e-20                      # the square underflows: y stays 0 beside eps
    x[2, 5] = 1e4                     # one value holds the row
    x[3, 130] = float("inf")
    x[4, 3] = float("nan")
    x[5] = torch.linspace(-3, 3, H)
    y, s, _, r = bd.maxsim_rmsnorm_fwd(x.to(DEV), out_dtype=torch.int8, with_rstd=True)
    y, s = y.cpu(), s.cpu()
    assert torch.all(y[0] == 0) and s[0] == 1
    assert y[2, 5] == 127 and torch.count_nonzero(y[2]) == 1
    assert torch.isnan(s[3]) and torch.isnan(s[4]) and torch.all(y[3:5] == 0)
    assert torch.isfinite(s[[0, 1, 2, 5]]).all()
    y, s, _, _ = bd.maxsim_rmsnorm_fwd(x.to(DEV), out_dtype=torch.float8_e4m3fn)
    y, s = y.float().cpu(), s.cpu()
    # an infinity: r = 0, so its block is not finite and the other block is 0
    assert torch.isnan(s[3, 1]) and s[3, 0] == 1 and torch.all(y[3] == 0)
    assert torch.isnan(s[4]).all()
    y, _, _, _ = bd.maxsim_rmsnorm_fwd(x.to(DEV))
    assert torch.isnan(y[4]).all() and torch.isnan(y[3, 130]) and torch.all(y[3, :130] == 0)
    # eps = 0 and a row of zeros: 0 / 0
    y, _, _, _ = bd.maxsim_rmsnorm_fwd(x[:1].to(DEV), eps=0.0)
    assert torch.isnan(y).all()


def test_no_rows(bd):
    x = torch.zeros(0, 64, device=DEV)
    y, s, _, r = bd.maxsim_rmsnorm_fwd(x, out_dtype=torch.int8, with_rstd=True)
    assert y.shape == (0, 64) and s.shape == (0,) and r.shape == (0,)
    dw = torch.full((64,), 7.0, device=DEV)
    dx, got = bd.maxsim_rmsnorm_bwd(x, x, torch.zeros(0, device=DEV), dweight=dw)
    assert dx.shape == (0, 64) and torch.all(got == 0)


def test_many_rows(bd):
    """More rows than one launch of the backward has workgroups, and an odd number of them."""
    R, H = 70001, 128
    x = torch.randn(R, H, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()
    y, s, _, r = bd.maxsim_rmsnorm_fwd(x, out_dtype=torch.int8, with_rstd=True)
    _, _, want = ref.rmsnorm(x.cpu(), None, None, 1e-6)
    ref.check_held(y, s[:, None], want, 1, H, "i8", ERR, "many")
    dx, dw = bd.maxsim_rmsnorm_bwd(x, x, r)
    _, want, _, size = ref.rmsnorm_bwd(x.cpu(), x.cpu(), r.cpu(), None, None)
    # a thread's chain: 70001 / (1024 groups * 16 rows) rows, 16 in a workgroup, 64 partial rows, 16 runs
    assert torch.all((dw.double().cpu() - want).abs() <= 2.0 ** -16 * size)


def test_int8_rows_feed_the_int8_scan(bd):
    """The int8 output is maxsim_fwd_i8's operand: scores equal those of the same codes scored by the oracle."""
    import oracle
    Q, D = rows(1, 2 * 32, 128, torch.float32).to(DEV), rows(2, 300, 128, torch.float32).to(DEV)
    q, qs, _, _ = bd.maxsim_rmsnorm_fwd(Q, out_dtype=torch.int8)
    d, ds, _, _ = bd.maxsim_rmsnorm_fwd(D, out_dtype=torch.int8)
    cu = torch.tensor([0, 100, 100, 171, 300], dtype=torch.int32, device=DEV)
    s, a = bd.maxsim_fwd_i8(q.reshape(2, 32, 128), qs.reshape(2, 32), d, ds, cu, 129)
    s_ref, a_ref = oracle.fwd_i8(q.cpu().numpy().reshape(2, 32, 128), qs.cpu().numpy().reshape(2, 32), d.cpu().numpy(),
                                 ds.cpu().numpy(), cu.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), s_ref) and np.array_equal(a.cpu().numpy(), a_ref)


def test_binding_refusals(bd):
    x = torch.zeros(4, 128, device=DEV)
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_fwd(x, torch.ones(127, device=DEV))
    with pytest.raises(TypeError):
        bd.maxsim_rmsnorm_fwd(x, torch.ones(128, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_fwd(x, residual=torch.zeros(5, 128, device=DEV))
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_fwd(x, residual=x[:1].expand(4, 128))
    with pytest.raises(TypeError):
        bd.maxsim_rmsnorm_fwd(x.int())
    with pytest.raises(TypeError):
        bd.maxsim_rmsnorm_fwd(x, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_fwd(x, scale=torch.ones(4, device=DEV))
    with pytest.raises(bd.MaxSimError):
        bd.maxsim_rmsnorm_fwd(torch.zeros(1, 32769, device=DEV))
    many = torch.zeros(5000, 128, device=DEV)
    with pytest.raises(bd.MaxSimError):
        bd.maxsim_rmsnorm_bwd(many, many, many[:, 0].contiguous(),
                              workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_bwd(x, x, torch.ones(3, device=DEV))
