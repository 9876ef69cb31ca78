"""Attention at the edges of what its calls allow, forward and backward, on the device.  Run on an MI355X: pytest -m gpu."""
import functools
import types

import pytest
import torch

import layers_ref as ref

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


# (queries, keys) of two sequences, query heads to a key head: few rows whole and in parts, many rows whole and in parts
FORMS = [([3, 2], [60, 9], 2), ([1, 1], [3000, 700], 4), ([90, 40], [90, 300], 2), ([150, 9], [4100, 3000], 2)]


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)], ids=str)
@pytest.mark.parametrize("nq,nk,G", FORMS, ids=str)
@pytest.mark.parametrize("where", ["q", "k", "v", "k inf", "g"])
def test_a_nan_reaches_the_rows_that_see_it(bd, where, nq, nk, G, D, dtype):
    """One NaN in the last query's row, in a key, in a value, in dO, or an infinite key: out, lse and gradients of the rows
    that see it are NaN, and the other sequence's stay as they were, bit for bit."""
    B, Lq, Lk, H = 2, max(nq), max(nk), 2 * G
    t = {"q": rand(B, Lq, H, D, dtype=dtype, seed=1), "k": rand(B, Lk, 2, D, dtype=dtype, seed=2),
         "v": rand(B, Lk, 2, D, dtype=dtype, seed=3), "g": rand(B, Lq, H, D, dtype=dtype, seed=4)}
    ints = lambda n: torch.tensor(n, dtype=torch.int32, device=DEV)  # noqa: E731
    how = dict(window=(-1, 0), q_lens=ints(nq), k_lens=ints(nk))

    def call():
        out, lse = bd.maxsim_attn_fwd(t["q"], t["k"], t["v"], with_lse=True, **how)
        return [out, lse, *bd.maxsim_attn_bwd(t["g"], t["q"], t["k"], t["v"], out, lse, **how)]

    clean = call()
    name = where[0]
    at = nq[0] - 1 if name in "qg" else nk[0] - nq[0]  # the key where the first query stands: all see it
    t[name][0, at, 1 if name in "kv" else G, 5] = INF if where == "k inf" else NAN  # heads G .. 2 G - 1 share key head 1
    out, lse, dq, dk, dv = got = call()
    for a, b in zip(got, clean):
        assert torch.equal(a[1], b[1])
        assert torch.equal(a[0, :, :G] if a.shape[2] == H else a[0, :, :1], b[0, :, :G] if b.shape[2] == H else b[0, :, :1])
    rows, heads = (slice(at, at + 1), slice(G, G + 1)) if name in "qg" else (slice(0, nq[0]), slice(G, H))
    none = lambda x: bool(torch.isnan(x).all())  # noqa: E731
    if name == "g":
        assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
        assert none(dq[0, at, G]) and none(dk[0, :nk[0], 1]) and none(dv[0, :nk[0], 1, 5])
        return
    if where == "k inf":  # scores of +infinity: NaN; of -infinity: a weight of 0
        up = torch.zeros(B, Lq, H, dtype=torch.bool, device=DEV)
        up[0, :nq[0], G:] = t["q"][0, :nq[0], G:, 5] > 0
        assert none(out[up]) and none(lse[up]) and none(dq[up])
        # of -infinity: the other keys' weights; a query that sees no other key (the first, at the infinite one) as one that sees none
        down = ~up[0, :nq[0], G:]
        alone = down & (torch.arange(nq[0], device=DEV) + at == 0)[:, None]
        l, o = lse[0, :nq[0], G:], out[0, :nq[0], G:]
        assert torch.all(l[alone] == -INF) and torch.all(o[alone] == 0)
        assert torch.isfinite(l[down & ~alone]).all() and torch.isfinite(o[down]).all()
        return
    if name == "v":
        assert none(out[0, rows, heads, 5]) and torch.isfinite(out[0, rows, heads, :5]).all() and torch.equal(lse, clean[1])
        assert none(dq[0, rows, heads]) and none(dk[0, at, 1]) and torch.equal(dv, clean[4])
    else:
        assert none(out[0, rows, heads]) and none(lse[0, rows, heads]) and none(dq[0, rows, heads])
        assert none(dk[0, at, 1]) and none(dv[0, at, 1])


@pytest.mark.parametrize("nq,Lk", [(1, 3000), (150, 4100)])
def test_a_nan_behind_a_weight_of_zero(bd, nq, Lk):
    """A value that is not finite times a weight that fell to 0 is NaN, in the parts' join too."""
    q, k, v = rand(1, nq, 2, 64), rand(1, Lk, 1, 64, seed=2), rand(1, Lk, 1, 64, seed=3)
    q[:], k[:], k[0, :400] = 1.0, 1.0, -100.0  # scores 8, and -800 through more than the first part
    v[0, 7, 0, 9] = NAN
    out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True)
    assert torch.isnan(out[..., 9]).all() and torch.isfinite(out[..., :9]).all() and torch.isfinite(lse).all()


def test_a_query_that_is_not_a_number_over_a_long_cache(bd):
    """Every score of the row is NaN, in every part."""
    q, k, v = rand(2, 1, 4, 64), rand(2, 9000, 1, 64, seed=2), rand(2, 9000, 1, 64, seed=3)
    q[0, 0, 2] = NAN
    out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True)
    assert torch.isnan(out[0, 0, 2]).all() and torch.isnan(lse[0, 0, 2])
    assert torch.isfinite(out[1]).all() and torch.isfinite(out[0, 0, [0, 1, 3]]).all()


def fp16_gradients(bd, t, window, scale, where, lens=None):
    """dQ, dK and dV of fp16 rows on the host, one sequence [L, H, D], within the 64-bit form's bounds, where what falls below fp16's
    values does so on the scale of a key's (or a row's) own largest dS: 2^-32 of it (2^-31, for the rounding of that largest)."""
    q, k, v, g = (t[n] for n in "qkvg")
    L, Hq, D = q.shape
    Hk, Lk = k.shape[1], k.shape[0]
    G = Hq // Hk
    want = ref.attention(q, k, v, [(0, L, 0, Lk)], scale, window, 0, g)
    vis = ref.seen(L, Lk, window, 0)
    dq, dk = want["dq"][1], want["dk"][1]
    for h in range(Hk):
        most, less = torch.zeros(Lk, dtype=torch.float64), torch.zeros(Lk, D, dtype=torch.float64)
        seen_q = torch.zeros(Lk, D, dtype=torch.float64)
        for j in range(h * G, (h + 1) * G):
            qd, kd, vd, gd = q[:, j].double(), k[:, h].double(), v[:, h].double(), g[:, j].double()
            p = torch.softmax((scale * qd @ kd.t()).masked_fill(~vis, -INF), 1)
            dp = gd @ vd.t()
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            top = gd.abs().amax(1, keepdim=True)
            low = vis.double() * 2.0 ** -25
            # the reference's terms of fp16's smallest values, in the scale of the rows' dO, give way to these
            dq[:, j] += scale * (2.0 ** -31 * ds.abs().amax(1, keepdim=True) * vis.double() - low * top) @ kd.abs()
            less += scale * (low * top.max()).t() @ qd.abs()
            most = torch.maximum(most, ds.abs().amax(0))
            seen_q += vis.double().t() @ qd.abs()
        dk[:, h] += scale * 2.0 ** -31 * most[:, None] * seen_q - less
    d = {n: x[None].to(DEV) for n, x in t.items()}
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], scale=scale, window=window, with_lse=True)
    ref.check(out, want["out"], where + " out")
    got = bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, scale=scale, window=window)
    for n, x in zip(("dq", "dk", "dv"), got):
        ref.check(x, want[n], where + " " + n)
    return got


@pytest.mark.parametrize("window", [(-1, 0), (-1, -1), (90, 0)], ids=str)
@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("r", [1, 12, 18])
def test_one_large_row_of_dout_in_fp16(bd, r, G, window):
    """An early row's dO is 2^r times the others': it takes nothing from the keys that it does not see, nor from those that
    it hardly looks at."""
    t = {n: torch.randn(1500, 2 * G if n in "qg" else 2, 64, generator=torch.Generator().manual_seed(i)).to(F16)
         for i, n in enumerate("qkvg")}
    t["g"] *= 2.0 ** -6
    t["g"][1, 0] *= 2.0 ** r
    fp16_gradients(bd, t, window, 0.125, str(r))


@pytest.mark.parametrize("window", [(-1, 0), (3, 0)], ids=str)
@pytest.mark.parametrize("vsize,gsize", [(200.0, 1.0), (8000.0, 2.0 ** -6), (8000.0, 2.0 ** -20), (2.0 ** -12, 2000.0)], ids=str)
def test_values_and_gradients_of_any_size_in_fp16(bd, vsize, gsize, window):
    """dO v^T of up to millions times what fp16 holds beside a row's dO, and far below its smallest values."""
    t = {n: torch.randn(300, 2, 64, generator=torch.Generator().manual_seed(i)) for i, n in enumerate("qkvg")}
    t["v"] *= vsize
    t["g"] *= gsize
    got = fp16_gradients(bd, {n: x.to(F16) for n, x in t.items()}, window, 0.125, "%g %g" % (vsize, gsize))
    assert all(torch.isfinite(x).all() for x in got)


def test_large_values_that_agree_with_dout_in_fp16(bd):
    """dO of one sign and v of either, a key's all the same: dO (v - out) is 128 columns times 30000 times dO."""
    t = {n: torch.randn(200, 1, 128, generator=torch.Generator().manual_seed(i)) for i, n in enumerate("qkvg")}
    t["v"] = torch.where(t["v"][..., :1] > 0, 30000.0, -30000.0).expand(200, 1, 128)
    t["g"] = torch.full((200, 1, 128), 2.0 ** -10)
    got = fp16_gradients(bd, {n: x.to(F16).contiguous() for n, x in t.items()}, (4, 2), 128 ** -0.5, "agree")
    assert all(torch.isfinite(x).all() for x in got)


@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 40)], ids=str)
@pytest.mark.parametrize("behind", ["large", "nan", "zeros", "anything"])
def test_an_lse_in_the_callers_own_memory(bd, behind, dtype, D, general):
    """A view of the forward's steps with something else behind its numbers: as a contiguous lse, or, where that happens to be
    as small as what rounding leaves, off by as much again."""
    if general:
        bd = types.SimpleNamespace(**{n: functools.partial(getattr(bd, n), stream=torch.cuda.current_stream())
                                      for n in ("maxsim_attn_fwd", "maxsim_attn_bwd")})
    t = {n: torch.randn(2 * 90, 4 if n in "qg" else 2, D, generator=torch.Generator().manual_seed(i)).to(dtype)
         for i, n in enumerate("qkvg")}
    d = {n: x.to(DEV).reshape(2, 90, -1, D) for n, x in t.items()}
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], window=(20, 0), with_lse=True)
    lens = [(0, 90, 0, 90), (90, 90, 90, 90)]
    exact, want = (ref.attention(t["q"], t["k"], t["v"], lens, D ** -0.5, (20, 0), 0, t["g"], exact_rest=e) for e in (True, False))
    plain = bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse.contiguous(), window=(20, 0))
    own = torch.randn(2, 90, 4, 1 + D // 2, generator=torch.Generator().manual_seed(9)).to(DEV)
    if behind != "anything":
        own.view(dtype).fill_({"large": 3.0, "nan": NAN, "zeros": 0.0}[behind])
    own[..., 0] = lse
    got = bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, own[..., 0], window=(20, 0))
    for n, a, b in zip(("dq", "dk", "dv"), got, plain):
        if behind != "anything":
            assert torch.equal(a, b), n
        ref.check(b, want[n], n)
        ref.check(a, (want[n][0], want[n][1] + 1.02 * (want[n][1] - exact[n][1])), n)


@pytest.mark.parametrize("at", [1, 4])
def test_autograd_of_rows_that_start_anywhere(bd, at):
    """Contiguous q, k, v and a contiguous dO whose memory starts 2 or 8 bytes off 16: the same bits as aligned ones."""
    def off(t):
        flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)
        return flat[at:at + t.numel()].copy_(t.flatten()).view(t.shape)

    q, k, v, g = (rand(2, 40, 4, 64, dtype=F16, seed=i) for i in range(4))
    want = torch.autograd.grad(bd.attention(*(x := [t.requires_grad_() for t in (q, k, v)]), window=(9, 0)), x, g)
    x = [off(t.detach()).requires_grad_() for t in (q, k, v)]
    assert x[0].is_contiguous() and x[0].data_ptr() % 16
    o = bd.attention(*x, window=(9, 0))
    assert torch.equal(o, bd.attention(q, k, v, window=(9, 0)))
    for a, b in zip(torch.autograd.grad(o, x, off(g)), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("nq,Lk", [(1, 600), (1, 65537), (150, 600), (150, 20001)])
def test_many_keys_of_small_weights_behind_a_first_token(bd, nq, Lk, dtype):
    """The first key's weight is 2^25.5 times each other's, which have all of the values: together they are 1 / 700 of the row
    at 65537 keys.  In fp16 a weight is held to half a step of 2^-31 of the largest."""
    q, k = torch.zeros(nq, 1, 64, dtype=dtype), torch.zeros(Lk, 1, 64, dtype=dtype)
    v = torch.randn(Lk, 1, 64, generator=torch.Generator().manual_seed(3)).abs().to(dtype)
    q[:], k[0], v[0] = 0.5, 17.6875 / 32, 0.0  # a score of 17.6875 (in bf16 17.75)
    want = ref.attention(q, k, v, [(0, nq, 0, Lk)], 1.0, (-1, -1), 0)
    if dtype == F16:
        want["out"][1][:] -= (2.0 ** -25 - 2.0 ** -32) * v.double().sum(0)
    out, lse = bd.maxsim_attn_fwd(*(t[None].to(DEV) for t in (q, k, v)), scale=1.0, with_lse=True)
    ref.check(out, want["out"], "out")
    ref.check(lse, want["lse"], "lse")


def test_starts_out_of_order(bd):
    """Starts that no caller should pass: rows that one sequence of them owns are that sequence's, though they lie past the
    last start or before the first; rows past all of them are zeros."""
    n = 90
    q, k, v, g = (rand(n, 2, 64, dtype=F16, seed=i) for i in range(4))
    for starts, a, b in (([20, 60, 40], 20, 60), ([50, 10, 40], 10, 40), ([70, 70, 5, 70], 5, 70)):
        cu = torch.tensor(starts, dtype=torch.int32, device=DEV)
        one = torch.tensor([a, b], dtype=torch.int32, device=DEV)
        got, want = [], []
        for to, c in ((got, cu), (want, one)):
            how = dict(cu_q=c, cu_k=c, max_q=n, max_k=n, window=(9, 0))
            out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True, **how)
            to += [out, lse, *bd.maxsim_attn_bwd(g, q, k, v, out, lse, **how)]
        for x, y in zip(got, want):
            assert torch.equal(x, y) and torch.all(x[:a] == 0) and torch.all(x[b:] == 0), starts


@pytest.mark.parametrize("window", [(-1, 0), (30, 5)], ids=str)
def test_many_short_sequences_in_fp16(bd, window):
    """More key tiles than CUs at a width of 128: two workgroups of dK and dV to a CU."""
    n = [1 + 13 * i % 120 for i in range(75)]
    t = {m: torch.randn(sum(n), 4, 128, generator=torch.Generator().manual_seed(i)).to(F16) for i, m in enumerate("qkvg")}
    cu = [0] + torch.tensor(n).cumsum(0).tolist()
    want = ref.attention(t["q"], t["k"], t["v"], [(a, m, a, m) for a, m in zip(cu, n)], 128 ** -0.5, window, 0, t["g"])
    d = {m: x.to(DEV) for m, x in t.items()}
    starts = torch.tensor(cu, dtype=torch.int32, device=DEV)
    how = dict(window=window, cu_q=starts, cu_k=starts, max_q=max(n), max_k=max(n))
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], with_lse=True, **how)
    got = dict(out=out, lse=lse, **dict(zip(("dq", "dk", "dv"), bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, **how))))
    for m in got:
        ref.check(got[m], want[m], m)
