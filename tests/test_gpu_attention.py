"""Attention with a sliding window and first tokens that stay visible, forward and backward, against its 64-bit form.
Run on an MI355X: pytest -m gpu."""
import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def rand(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)


def case(dtype, nq, nk, Hq, Hk, D, window=(-1, -1), sinks=0, packed=False, train=False, more=0, Lq=None, Lk=None, size=1.0,
         gsize=1.0):
    """Inputs on the host: sequences of nq[b] queries and nk[b] keys; `more` rows behind the last packed one."""
    B = len(nq)
    if packed:
        rq, rk = sum(nq) + more, sum(nk) + more
        lens, a, b = [], 0, 0
        for i, j in zip(nq, nk):
            lens.append((a, i, b, j))
            a, b = a + i, b + j
    else:
        Lq, Lk = Lq or max(nq), Lk or max(nk)
        rq, rk = B * Lq, B * Lk
        lens = [(b * Lq, nq[b], b * Lk, nk[b]) for b in range(B)]
    t = {"q": rand(rq, Hq, D, dtype=dtype, seed=1) * size, "k": rand(rk, Hk, D, dtype=dtype, seed=2),
         "v": rand(rk, Hk, D, dtype=dtype, seed=3)}
    if train:
        t["g"] = (rand(rq, Hq, D, dtype=torch.float32, seed=4) * gsize).to(dtype)
    return dict(t=t, lens=lens, nq=nq, nk=nk, packed=packed, window=window, sinks=sinks, Lq=Lq, Lk=Lk, D=D)


def device_args(c):
    B = len(c["nq"])
    how = dict(window=c["window"], sinks=c["sinks"])
    shape = lambda t, L: t.to(DEV) if c["packed"] else t.to(DEV).reshape((B, L) + t.shape[1:])  # noqa: E731
    d = {n: shape(t, c["Lq"] if n in "qg" else c["Lk"]) for n, t in c["t"].items()}
    if c["packed"]:
        how.update(cu_q=cu_of(c["nq"]).to(DEV), cu_k=cu_of(c["nk"]).to(DEV), max_q=max(c["nq"]), max_k=max(c["nk"]))
    else:
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        how.update(q_lens=None if min(c["nq"]) == c["Lq"] else ints(c["nq"]),
                   k_lens=None if min(c["nk"]) == c["Lk"] else ints(c["nk"]))
    return d, how


def run(bd, c, scale=None, where=""):
    d, how = device_args(c)
    t = c["t"]
    want = ref.attention(t["q"], t["k"], t["v"], c["lens"], scale or c["D"] ** -0.5, c["window"], c["sinks"], t.get("g"))
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], scale=scale, with_lse=True, **how)
    ref.check(out, want["out"], where + " out")
    ref.check(lse, want["lse"], where + " lse")
    got = [out, lse]
    if "g" in d:
        grads = bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, scale=scale, **how)
        for n, g in zip(("dq", "dk", "dv"), grads):
            ref.check(g, want[n], where + " " + n)
        got += grads
    return got


WINDOWS = [((-1, -1), 0), ((-1, 0), 0), ((7, 0), 0), ((7, 0), 3), ((16, 16), 1), ((0, 0), 0), ((0, 5), 70), ((40, -1), 2),
           ((100, 3), 200)]


@pytest.mark.parametrize("window,sinks", WINDOWS, ids=str)
@pytest.mark.parametrize("dtype,D", [(F16, 64), (BF16, 128)], ids=str)
def test_windows(bd, dtype, D, window, sinks):
    """Documents of one token to some hundred, packed, none of a tile's size."""
    n = [1, 33, 0, 130, 257, 2]
    run(bd, case(dtype, n, n, 4, 2, D, window, sinks, packed=True, train=True))


@pytest.mark.parametrize("D", [8, 16, 40, 56, 64, 72, 80, 96, 112, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
def test_widths(bd, dtype, D):
    run(bd, case(dtype, [70, 45], [70, 45], 3, 1, D, (20, 0), 2, train=True))


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 5), (12, 4), (8, 1), (7, 1), (40, 1), (33, 3)])
def test_shared_heads(bd, Hq, Hk):
    run(bd, case(BF16, [50, 9], [50, 9], Hq, Hk, 64, (30, 0), 1, packed=True, train=True))


@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((-1, 0), 0), ((50, 0), 4), ((10, 10), 0)], ids=str)
@pytest.mark.parametrize("nq,nk", [([1] * 5, [1, 700, 33, 0, 64]), ([4, 0, 9, 9, 1], [90, 200, 9, 300, 1]), ([150, 40], [600, 601]),
                                   ([60, 33], [20, 0])], ids=str)
@pytest.mark.parametrize("G", [1, 4])
def test_queries_at_the_end_of_their_keys(bd, nq, nk, window, sinks, G):
    """Next tokens, some tokens against a cache, and more queries than keys: the first ones then see nothing."""
    run(bd, case(BF16, nq, nk, 2 * G, 2, 64, window, sinks, train=True, Lk=max(nk) + 5))


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)], ids=str)
@pytest.mark.parametrize("nq", [1, 7, 130])
@pytest.mark.parametrize("window,sinks", [((-1, 0), 0), ((1500, 0), 4)], ids=str)
def test_a_long_cache_in_parts(bd, D, dtype, nq, window, sinks):
    """Keys split over workgroups and joined; one cache is short, so that some parts have no keys."""
    run(bd, case(dtype, [nq, nq, 1], [5003, 100, 4096], 4, 2, D, window, sinks))


def test_rows_that_see_nothing(bd):
    c = case(F16, [40, 3], [10, 0], 2, 2, 64, (-1, 0), 0, train=True)
    out, lse, dq, dk, dv = run(bd, c)
    assert torch.all(out[0, :30] == 0) and torch.all(lse[0, :30] == -float("inf")) and torch.all(dq[0, :30] == 0)
    assert torch.all(out[1] == 0) and torch.all(dk[1] == 0) and torch.all(dv[1] == 0)


@pytest.mark.parametrize("packed", [False, True])
def test_what_lies_past_the_sequences(bd, packed):
    """Rows of no sequence hold NaN: nothing of them is read.  In outputs made by the call they are zeros, in given ones
    they stay."""
    n = [20, 0, 71]
    c = case(BF16, n, n, 4, 2, 64, (30, 30), 1, packed=packed, train=True, more=45, Lq=80, Lk=90)
    d, how = device_args(c)
    mark = {}
    for name, L in (("q", 80), ("k", 90), ("v", 90), ("g", 80)):
        keep = torch.zeros(c["t"][name].shape[0], dtype=torch.bool)
        for q0, nq, k0, nk in c["lens"]:
            a, m = (q0, nq) if name in "qg" else (k0, nk)
            keep[a:a + m] = True
        mark[name] = keep.to(DEV).reshape(d[name].shape[:-2])
    clean = run(bd, c)
    for name in d:
        d[name][~mark[name]] = float("nan")
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], with_lse=True, **how)
    grads = bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, **how)
    for a, b in zip([out, lse] + list(grads), clean):
        assert torch.equal(a, b)
    for t, m in zip([out, lse] + list(grads), "qqqkk"):
        assert torch.all(t[~mark[m]] == 0)
    filled = [torch.full_like(t.contiguous(), 5.0) for t in [out, lse] + list(grads)]
    bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], out=filled[0], lse=filled[1], **how)
    bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, dq=filled[2], dk=filled[3], dv=filled[4], **how)
    for a, b, m in zip(filled, clean, "qqqkk"):
        assert torch.equal(a[mark[m]], b[mark[m]]) and torch.all(a[~mark[m]] == 5)


def test_lengths_out_of_range_stay_inside(bd):
    """Lengths and starts that no caller should pass: cut to the memory, as documented; what is in range is right."""
    c = case(BF16, [30, 30], [30, 30], 2, 1, 64)
    d, _ = device_args(c)
    want, _ = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"])
    lens = torch.tensor([1 << 30, -7], dtype=torch.int32, device=DEV)
    out, _ = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], q_lens=lens, k_lens=lens)
    assert torch.equal(out[0], want[0]) and torch.all(out[1] == 0)
    flat = {n: t.flatten(0, 1) for n, t in d.items()}
    cu = torch.tensor([0, 30, 1 << 30], dtype=torch.int32, device=DEV)
    out, _ = bd.maxsim_attn_fwd(flat["q"], flat["k"], flat["v"], cu_q=cu, cu_k=cu, max_q=30, max_k=30)
    assert torch.equal(out, want.flatten(0, 1))
    cu = torch.tensor([-5, 30, 10], dtype=torch.int32, device=DEV)
    out, _ = bd.maxsim_attn_fwd(flat["q"], flat["k"], flat["v"], cu_q=cu, cu_k=cu, max_q=30, max_k=30)
    assert torch.equal(out[:30], want[0])


def test_scores_of_any_size(bd):
    """Scores from a thousandth to hundreds: the softmax is flat, or one key's alone."""
    for size in (1e-3, 30.0):
        for dtype in (F16, BF16):
            run(bd, case(dtype, [90], [90], 2, 2, 64, (-1, 0), 0, train=True, size=size), where=str(size))
    run(bd, case(F16, [65], [300], 2, 1, 128, (-1, -1), 0, train=True), scale=1.5)


@pytest.mark.parametrize("gsize", [1e-6, 3e-4, 300.0])
def test_gradients_of_any_size_in_fp16(bd, gsize):
    """Attention over 1500 keys is flat: P near 1 / 1500, dS far below fp16's normal values."""
    run(bd, case(F16, [40, 1500], [40, 1500], 2, 1, 64, (-1, -1), 0, train=True, size=0.1, gsize=gsize))


def test_gradients_of_rows_of_different_sizes_in_fp16(bd):
    """Rows of dO that grow by 2^20 along a sequence: each product is in the scale of the largest so far."""
    c = case(F16, [300], [300], 2, 2, 64, (-1, 0), 0, train=True)
    grow = torch.exp2(torch.linspace(-14, 6, 300))[:, None, None]
    c["t"]["g"] = (c["t"]["g"].float() * grow).to(F16)
    run(bd, c)
    c["t"]["g"] = c["t"]["g"].flip(0)
    run(bd, c)
    c["t"]["g"][100:200] = 0
    run(bd, c)


def test_heads_before_tokens_and_a_fused_projection(bd):
    """[B, H, L, D] storage, and q, k, v as slices of one projection: the same values as contiguous ones, bit for bit."""
    c = case(BF16, [77, 77], [77, 77], 6, 2, 64, (20, 0), 1, train=True)
    d, how = device_args(c)
    want = run(bd, c)
    moved = {n: t.transpose(1, 2).contiguous().transpose(1, 2) for n, t in d.items()}
    out, lse = bd.maxsim_attn_fwd(moved["q"], moved["k"], moved["v"], with_lse=True, **how)
    got = [out, lse] + list(bd.maxsim_attn_bwd(moved["g"], moved["q"], moved["k"], moved["v"], out, lse, **how))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    fused = torch.cat([d["q"], d["k"], d["v"]], 2)
    out, _ = bd.maxsim_attn_fwd(fused[:, :, :6], fused[:, :, 6:8], fused[:, :, 8:], **how)
    assert torch.equal(out, want[0])
    # outputs in slices of wider memory
    wide = torch.full((2, 77, 10, 64), 3.0, dtype=BF16, device=DEV)
    bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], want[0], want[1], dq=wide[:, :, :6], dk=wide[:, :, 6:8], dv=wide[:, :, 8:], **how)
    assert torch.equal(wide, torch.cat(want[2:], 2))


def test_a_broadcast_cache(bd):
    """One prefix for all sequences, and one head for all: steps of 0."""
    c = case(BF16, [3, 3, 3], [200, 200, 200], 4, 4, 64)
    d, how = device_args(c)
    k, v = d["k"][:1, :, :1].expand(3, 200, 4, 64), d["v"][:1, :, :1].expand(3, 200, 4, 64)
    a, _ = bd.maxsim_attn_fwd(d["q"], k, v, **how)
    b, _ = bd.maxsim_attn_fwd(d["q"], k.contiguous(), v.contiguous(), **how)
    assert torch.equal(a, b)


def test_offsets_past_32_bits(bd):
    """A cache whose rows lie 128 KB apart, 9 GB in all, and more bytes than 2^32 between a sequence's first and last key."""
    L, step = 70001, 65536
    big = torch.empty(L * step, dtype=BF16, device=DEV)
    flat = rand(L, 3, 64, dtype=BF16, seed=5)
    k, v = (big[64 * i:].as_strided((1, L, 1, 64), (0, step, 64, 1)) for i in (0, 2))
    k.copy_(flat[None, :, :1].to(DEV))
    v.copy_(flat[None, :, 1:2].to(DEV))
    q = rand(1, 200, 2, 64, dtype=BF16, seed=6).to(DEV)
    for nq, window, sinks in ((1, (-1, 0), 0), (200, (500, 0), 4), (200, (-1, 0), 0)):
        qs = q[:, :nq]
        got, _ = bd.maxsim_attn_fwd(qs, k, v, window=window, sinks=sinks)
        want, _ = bd.maxsim_attn_fwd(qs, k.contiguous(), v.contiguous(), window=window, sinks=sinks)
        assert torch.equal(got, want)
    del big


def test_one_call_again_and_again(bd):
    """The same bits each time: forward, in parts, and backward."""
    c = case(BF16, [300, 300], [300, 300], 4, 1, 128, (64, 0), 2, train=True)
    a, b = run(bd, c), run(bd, c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = case(BF16, [1], [9000], 4, 1, 128)
    assert torch.equal(run(bd, c)[0], run(bd, c)[0])


def test_gradient_by_differences(bd):
    """Along a direction of q, k and v: the 64-bit form's difference quotient, with the kernel's bounds."""
    c = case(F16, [37], [37], 4, 2, 40, (9, 0), 2, train=True)
    t = c["t"]
    got = run(bd, c)
    dirs = [rand(*t[n].shape, dtype=torch.float32, seed=10 + i).double() for i, n in enumerate("qkv")]

    def value(e):
        x = [t[n].double() + e * d for n, d in zip("qkv", dirs)]
        out = torch.zeros_like(x[0])
        vis = ref.seen(37, 37, c["window"], c["sinks"])
        for h in range(4):
            s = (x[0][:, h] @ x[1][:, h // 2].t() * 40 ** -0.5).masked_fill(~vis, -float("inf"))
            out[:, h] = torch.softmax(s, 1) @ x[2][:, h // 2]
        return (out * t["g"].double()).sum()

    slope = lambda e: (value(e) - value(-e)) / (2 * e)  # noqa: E731
    slopes = slope(1e-4), slope(2e-4)
    want = ref.attention(t["q"], t["k"], t["v"], c["lens"], 40 ** -0.5, c["window"], c["sinks"], t["g"])
    along = sum((g.double().cpu().reshape(d.shape) * d).sum() for g, d in zip(got[2:], dirs))
    bound = sum((want[n][1] * d.abs()).sum() for n, d in zip(("dq", "dk", "dv"), dirs))
    # the quotient's own error falls with e^2: a third of what the step's doubling changes
    assert abs(slopes[0] - along) <= bound + abs(slopes[1] - slopes[0]) + 1e-7


def test_an_lse_without_what_rounding_left(bd):
    """A contiguous lse does for the backward too, within the bound of a rounded out."""
    c = case(BF16, [90, 40], [90, 40], 4, 2, 64, (20, 0), 1, train=True)
    d, how = device_args(c)
    t = c["t"]
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], with_lse=True, **how)
    assert not lse.is_contiguous()
    want = ref.attention(t["q"], t["k"], t["v"], c["lens"], 64 ** -0.5, c["window"], c["sinks"], t["g"], exact_rest=False)
    grads = bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse.contiguous(), **how)
    for n, g in zip(("dq", "dk", "dv"), grads):
        ref.check(g, want[n], n)


def test_autograd(bd):
    """attention(): gradients of views of any layout, of broadcast keys, and of some inputs only."""
    c = case(BF16, [50, 50], [50, 50], 4, 2, 24, (20, 0), 1, train=True)
    d, how = device_args(c)
    _, _, dq, dk, dv = run(bd, c)
    wide = torch.cat([d["q"], d["k"], d["v"]], 2).requires_grad_()
    o = bd.attention(wide[:, :, :4], wide[:, :, 4:6], wide[:, :, 6:], **how)
    g, = torch.autograd.grad(o, wide, d["g"])
    assert torch.equal(g, torch.cat([dq, dk, dv], 2))
    odd = [t.transpose(-1, -2).contiguous().transpose(-1, -2).detach().requires_grad_(i != 1) for i, t in
           enumerate((d["q"], d["k"], d["v"]))]
    o = bd.attention(*odd, **how)
    got = torch.autograd.grad(o, (odd[0], odd[2]), d["g"].transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(got[0], dq) and torch.equal(got[1], dv)
    one = d["k"][:1].detach().requires_grad_()
    o = bd.attention(d["q"], one.expand(2, -1, -1, -1), d["v"], **how)
    got, = torch.autograd.grad(o, one, d["g"])
    full, = torch.autograd.grad(bd.attention(d["q"], (k2 := one.detach().expand(2, -1, -1, -1).contiguous().requires_grad_()),
                                             d["v"], **how), k2, d["g"])
    assert torch.equal(got, full.sum(0, keepdim=True))
    with torch.no_grad():
        assert torch.equal(bd.attention(d["q"], d["k"], d["v"], **how), run(bd, c)[0])


def test_packed_queries_against_a_padded_cache(bd):
    """The queries' layout and the keys' are independent: packed new tokens against a cache with room left, and the other way."""
    c = case(BF16, [3, 0, 9, 1], [40, 77, 9, 130], 4, 2, 64, (50, 0), 2, train=True, Lk=150)
    d, how = device_args(c)
    want = run(bd, c)
    nq, nk, lq = torch.tensor(c["nq"]), torch.tensor(c["nk"]), c["Lq"]
    q_rows = torch.cat([torch.arange(n) + b * lq for b, n in enumerate(c["nq"])]).to(DEV)
    k_rows = torch.cat([torch.arange(n) + b * 150 for b, n in enumerate(c["nk"])]).to(DEV)
    pick = lambda t, rows: t.flatten(0, 1)[rows].contiguous()  # noqa: E731
    how = dict(window=(50, 0), sinks=2)
    for packed_q in (True, False):
        q, g = (pick(d[n], q_rows) if packed_q else d[n] for n in "qg")
        k, v = (d[n] if packed_q else pick(d[n], k_rows) for n in "kv")
        lens = dict(cu_q=cu_of(c["nq"]).to(DEV), max_q=9, k_lens=nk.to(torch.int32).to(DEV)) if packed_q else \
            dict(q_lens=nq.to(torch.int32).to(DEV), cu_k=cu_of(c["nk"]).to(DEV), max_k=130)
        out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True, **how, **lens)
        got = [out, lse] + list(bd.maxsim_attn_bwd(g, q, k, v, out, lse, **how, **lens))
        for a, b, m in zip(got, want, "qqqkk"):
            if (m == "q") == packed_q:
                b = pick(b, q_rows if m == "q" else k_rows)
            assert torch.equal(a, b), m


@pytest.mark.parametrize("G,B,L", [(4, 1, 700), (3, 9, 300), (1, 2, 900), (8, 1, 40)])
def test_few_key_tiles_share_out_their_query_heads(bd, G, B, L):
    """dK and dV in parts: of query heads, and of far queries of the first tokens; with one query head in none."""
    n = [L] + [max(1, L // (i + 2)) for i in range(B - 1)]
    run(bd, case(BF16, n, n, 2 * G, 2, 128, (60, 0), 3, packed=True, train=True))
    run(bd, case(F16, n, n, G, 1, 64, (-1, -1), 0, train=True))


def test_first_tokens_past_a_key_tile(bd):
    """More first tokens than a tile of keys, and as many as the split allows, over sequences much longer than the window."""
    for sinks in (130, 256, 257):
        run(bd, case(BF16, [900, 131], [900, 131], 2, 1, 64, (20, 0), sinks, packed=True, train=True))
    run(bd, case(BF16, [500], [900], 2, 2, 64, (20, 5), 9, train=True))
    run(bd, case(F16, [900], [500], 2, 2, 64, (20, 5), 9, train=True))


def test_more_query_sequences_than_fit_a_round_of_xcds(bd):
    """Numbers of (sequence, key head) pairs that are dealt out over the XCDs in turn, in runs, and with a rest."""
    for B, Hk in ((9, 1), (8, 1), (65, 1), (13, 5), (3, 1)):
        n = [1 + (7 * i) % 60 for i in range(B)]
        run(bd, case(BF16, n, n, Hk, Hk, 16, (9, 9), 1, packed=True, train=True))


@pytest.mark.parametrize("seed", range(40))
def test_seeded_random_calls(bd, seed):
    """Sizes, layouts, windows and head counts by a seed, forward and backward within their bounds."""
    import random
    r = random.Random(seed)
    Hk = r.choice([1, 1, 2, 3])
    packed = r.random() < 0.5
    nk = [r.choice([0, 1, r.randint(1, 60), r.randint(1, 330)]) for _ in range(r.choice([1, 2, 5]))]
    if max(nk) == 0:
        nk[0] = 17
    kind = r.choice(["same", "same", "fewer", "any"])
    nq = [n if kind == "same" else r.randint(0, n) if kind == "fewer" else r.randint(0, 200) for n in nk]
    if max(nq) == 0:
        nq[0] = 1
    window = (r.choice([-1, 0, r.randint(1, 30), r.randint(1, 300)]), r.choice([-1, 0, 0, r.randint(1, 100)]))
    c = case(r.choice([F16, BF16]), nq, nk, Hk * r.choice([1, 2, 5]), Hk, 8 * r.randint(1, 16), window,
             r.choice([0, 1, 4, 40, 300]), packed=packed, train=True, more=r.choice([0, 3]), size=r.choice([0.3, 1.0, 3.0]))
    if not packed:
        c = case(c["t"]["q"].dtype, nq, nk, c["t"]["q"].shape[1], Hk, c["D"], window, c["sinks"], train=True,
                 Lq=max(nq) + r.choice([0, 2]), Lk=max(nk) + r.choice([0, 70]))
    run(bd, c, where="seed %d" % seed)


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)], ids=str)
@pytest.mark.parametrize("nq,nk,window,sinks", [([1, 1], [700, 40], (30, 0), 4), ([1, 1], [5000, 90], (40, 0), 3), ([5, 150], [300, 400], (20, 3), 2),
                                                ([40, 200], [400, 230], (9, 0), 0), ([3, 140], [90, 900], (5, 5), 130),
                                                ([30, 150], [300, 200], (60, 0), 1)], ids=str)
def test_keys_that_no_query_sees_may_hold_anything(bd, nq, nk, window, sinks, G, D, dtype):
    """A cache's dropped entries, between the first tokens and the window: NaN there changes no bit, and their
    gradients are 0."""
    c = case(dtype, nq, nk, 2 * G, 2, D, window, sinks, packed=True, train=True)
    want = run(bd, c)
    hidden = torch.zeros(sum(nk), dtype=torch.bool)
    for q0, n, k0, m in c["lens"]:
        hidden[k0:k0 + m] = ~ref.seen(n, m, window, sinks).any(0)
    assert hidden.any()
    c["t"]["k"][hidden] = float("nan")
    c["t"]["v"][hidden] = float("inf")
    d, how = device_args(c)
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], with_lse=True, **how)
    got = [out, lse] + list(bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, **how))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.all(got[3][hidden.to(DEV)] == 0) and torch.all(got[4][hidden.to(DEV)] == 0)


def test_some_of_the_packed_sequences(bd):
    """A part of the starts with all of the rows: the other sequences' rows are of no sequence, before and behind."""
    n = [40, 7, 133, 20, 5]
    c = case(BF16, n, n, 4, 2, 64, (30, 0), 1, packed=True, train=True)
    want = run(bd, c)
    d, how = device_args(c)
    how.update(cu_q=how["cu_q"][1:4].contiguous(), cu_k=how["cu_k"][1:4].contiguous())
    out, lse = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], with_lse=True, **how)
    got = [out, lse] + list(bd.maxsim_attn_bwd(d["g"], d["q"], d["k"], d["v"], out, lse, **how))
    one = bd.maxsim_attn_fwd(d["q"], d["k"], d["v"], **{**how, "max_q": 7, "max_k": 133,
                             "cu_q": how["cu_q"][:2].contiguous(), "cu_k": how["cu_k"][:2].contiguous()})[0]
    for a, b in zip(got, want):
        assert torch.equal(a[40:180], b[40:180]) and torch.all(a[:40] == 0) and torch.all(a[180:] == 0)
    assert torch.equal(one[40:47], want[0][40:47]) and torch.all(one[:40] == 0) and torch.all(one[47:] == 0)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
def test_first_tokens_of_a_long_sequence_with_a_narrow_window(bd, dtype):
    """Far queries in as many parts as there may be, which are longer than the window then."""
    run(bd, case(dtype, [9001], [9001], 1, 1, 16, (2, 0), 140, train=True))


@pytest.mark.parametrize("D,dtype,Lk,parts", [(64, F16, 4100, 16), (128, BF16, 4100, 16), (96, BF16, 2400, 9), (64, BF16, 2100, 8)], ids=str)
def test_keys_in_eight_to_sixteen_parts(bd, D, dtype, Lk, parts):
    """The join's other forms: four rows to a workgroup, and eight."""
    nq, nk = [64, 33, 0, 1], [Lk, 700, 300, 2000]
    c = case(dtype, nq, nk, 8, 2, D, (-1, 0), 0)
    d, how = device_args(c)
    a = bd._attn(d["q"], d["k"], d["v"], None, None, how["window"], 0, how["q_lens"], how["k_lens"], None, None, None, None)
    assert bd.lib().maxsim_attn_fwd_workspace_bytes(bd.ctypes.byref(a)) == parts * 4 * 64 * 8 * (D + 2) * 4
    run(bd, c)
