"""The attention layer's operators and the distillation loss as they are used: one after the other from projected rows to
MaxSim's scores, the loss and back; captured and replayed; on streams of their own; through either way of the binding.
Run on an MI355X: pytest -m gpu."""
import math

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


def rand(*shape, dtype=F16, seed=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


HOW = dict(window=(24, 24), sinks=1)


def rows_of(bd, fused, f, heads, **lengths):
    """Token rows [.., 128] from a projection's [.., 4 heads of 64]: q of `heads`, k and v of one each."""
    turned = bd.rope(fused[..., :heads + 1, :], f)
    o = bd.attention(turned[..., :heads, :], turned[..., heads:, :], fused[..., heads + 1:, :], **HOW, **lengths)
    return o.flatten(-2)


def test_from_projected_rows_to_the_loss_and_back(bd):
    """6 queries of 32 tokens and 10 padded documents through rotary positions, attention, MaxSim and the loss; every
    link's result within its own bounds, and autograd's gradients those of the calls one after the other."""
    f, _ = bd.rope_frequencies(64, device=DEV)
    lens = torch.tensor([100, 37, 64, 100, 1, 99, 80, 20, 55, 100], dtype=torch.int32, device=DEV)
    Q = rand(6, 32, 4, 64, seed=1).requires_grad_()
    D = rand(10, 100, 4, 64, seed=2).requires_grad_()
    index = torch.stack([torch.randperm(10, generator=torch.Generator().manual_seed(i))[:4] for i in range(6)]).to(torch.int32).to(DEV)
    teacher = rand(6, 4, dtype=torch.float32, seed=3)
    rows_q = rows_of(bd, Q, f, 2)
    rows_d = rows_of(bd, D, f, 2, q_lens=lens, k_lens=lens)
    cu = torch.arange(0, 1001, 100, dtype=torch.int32, device=DEV)
    scores = bd.maxsim(rows_q, rows_d.reshape(1000, 128), cu, 100)
    loss = bd.distill_loss(scores, index, teacher, temperature=2.0)
    gq, gd = torch.autograd.grad(loss.sum(), (Q, D))

    ones = torch.ones(6, device=DEV)
    want = ref.distill(scores.detach().cpu(), index.cpu(), teacher.cpu(), 2.0, ones.cpu())
    ref.check(loss.detach(), want["loss"], "loss")
    got_loss, stat = bd.maxsim_distill_fwd(scores.detach(), index, teacher, temperature=2.0)
    ds = bd.maxsim_distill_bwd(ones, scores.detach(), stat, index, teacher, temperature=2.0)
    ref.check(ds, want["dscores"], "dscores")
    _, argmax = bd.maxsim_fwd_varlen(rows_q.detach(), rows_d.detach().reshape(1000, 128), cu, 100)
    dq_rows, dd_rows, _, _ = bd.maxsim_bwd_varlen(rows_q.detach(), rows_d.detach().reshape(1000, 128), cu, 100, argmax, ds)
    for x, rows, d_rows, got, n, more in ((Q.detach(), rows_q, dq_rows, gq, [32] * 6, {}),
                                          (D.detach(), rows_d, dd_rows, gd, lens.tolist(), dict(q_lens=lens, k_lens=lens))):
        B, L = x.shape[:2]
        turned = bd.maxsim_rope(x[..., :3, :], f)
        at = torch.arange(L).repeat(B)
        ref.check(turned, ref.rope(x[..., :3, :].cpu().reshape(-1, 3, 64), f.cpu(), at, "half", 1.0), "rope")
        q, k, v = turned[..., :2, :], turned[..., 2:, :], x[..., 3:, :]
        g = d_rows.to(F16).reshape(B, L, 2, 64)
        flat = [t.cpu().reshape(B * L, -1, 64) for t in (q, k, v, g)]
        w = ref.attention(*flat[:3], [(b * L, n[b], b * L, n[b]) for b in range(B)], 0.125, HOW["window"], HOW["sinks"], flat[3])
        out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True, **HOW, **more)
        assert torch.equal(out.flatten(-2), rows)
        ref.check(out, w["out"], "out")
        dq, dk, dv = bd.maxsim_attn_bwd(g, q, k, v, out, lse, **HOW, **more)
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            ref.check(t, w[name], name)
        back = bd.maxsim_rope(torch.cat([dq, dk], 2), f, inverse=True)
        assert torch.equal(got, torch.cat([back, dv], 2))
    assert torch.all(gd[4, 1:] == 0) and torch.isfinite(gd).all() and torch.any(gd[0] != 0)


def step(bd, s):
    """One pass through every operator from the state's buffers."""
    x = bd.maxsim_rope(s["x"], s["f"], offsets=s["off"], layout="interleaved")
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True, **s["how"])
    grads = bd.maxsim_attn_bwd(s["g"], q, k, v, out, lse, **s["how"])
    nxt, _ = bd.maxsim_attn_fwd(s["q1"], s["cache"], s["cache"], k_lens=s["n"], window=(-1, 0))
    loss, stat = bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"])
    return [x, out, lse, *grads, nxt, loss, bd.maxsim_distill_bwd(s["w"], s["z"], stat, s["index"], s["teacher"])]


def state(bd, seed):
    n = torch.tensor([90, 33], dtype=torch.int32, device=DEV)
    return dict(x=rand(2, 90, 8, 64, dtype=BF16, seed=seed), f=bd.rope_frequencies(64, device=DEV)[0],
                off=torch.tensor([0, seed], dtype=torch.int32, device=DEV), g=rand(2, 90, 4, 64, dtype=BF16, seed=seed + 1),
                how=dict(window=(20, 0), sinks=2, q_lens=n, k_lens=n), q1=rand(2, 1, 4, 64, dtype=BF16, seed=seed + 2),
                cache=rand(2, 9000, 1, 64, dtype=BF16, seed=seed + 3), n=torch.tensor([9000, 100 * seed], dtype=torch.int32, device=DEV),
                z=rand(3, 20000, dtype=torch.float32, seed=seed + 4), teacher=rand(3, 7, dtype=torch.float32, seed=seed + 5),
                index=torch.randint(0, 20000, (3, 7), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)),
                w=rand(3, dtype=torch.float32, seed=seed + 6))


def fill(s, other):
    for n, t in s.items():
        if torch.is_tensor(t):
            t.copy_(other[n])
    for n in ("q_lens", "k_lens"):
        s["how"][n].copy_(other["how"][n])


def test_captured_and_replayed(bd):
    """One graph, replayed over inputs that change, with the program's own work between; each replay as the eager calls."""
    s = state(bd, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(bd, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(bd, s)
    for seed in (5, 9, 3, 7):
        other = state(bd, seed)
        fill(s, other)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step(bd, other)):
            assert torch.equal(a, b)
        junk = rand(1000, 1000, dtype=torch.float32) @ rand(1000, 1000, dtype=torch.float32)
        torch.cuda.synchronize()
        del junk


def test_two_streams_at_once_and_a_given_stream(bd):
    states, want = [state(bd, i) for i in (2, 4)], []
    for s in states:
        want.append(step(bd, s))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in states], []
    for _ in range(3):
        got = []
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                got.append(step(bd, s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    s = states[0]
    out, _ = bd.maxsim_attn_fwd(s["q1"], s["cache"], s["cache"], k_lens=s["n"], window=(-1, 0), stream=streams[0])
    x = bd.maxsim_rope(s["x"], s["f"], offsets=s["off"], layout="interleaved", stream=streams[1])
    loss, stat = bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"], stream=streams[0])
    d = bd.maxsim_distill_bwd(s["w"], s["z"], stat, s["index"], s["teacher"], stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][6]) and torch.equal(x, want[0][0]) and torch.equal(loss, want[0][7]) and torch.equal(d, want[0][8])


def test_given_workspaces(bd):
    """A workspace that the caller keeps; one too small is refused."""
    s = state(bd, 6)
    want, _ = bd.maxsim_attn_fwd(s["q1"], s["cache"], s["cache"], k_lens=s["n"], window=(-1, 0))
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        got, _ = bd.maxsim_attn_fwd(s["q1"], s["cache"], s["cache"], k_lens=s["n"], window=(-1, 0), workspace=ws)
        assert torch.equal(got, want)
    with pytest.raises(bd.MaxSimError) as e:
        bd.maxsim_attn_fwd(s["q1"], s["cache"], s["cache"], k_lens=s["n"], window=(-1, 0), workspace=ws[:256])
    assert e.value.status == bd.MAXSIM_ERR_WORKSPACE
    loss, _ = bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"], workspace=ws)
    assert torch.equal(loss, bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"])[0])


def test_no_sequences(bd):
    e = torch.empty
    q = e(0, 5, 4, 64, dtype=BF16, device=DEV)
    out, lse = bd.maxsim_attn_fwd(q, q, q, with_lse=True)
    assert out.shape == q.shape and [t.shape for t in bd.maxsim_attn_bwd(q, q, q, q, out, lse)] == [q.shape] * 3
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    flat = rand(7, 4, 64, dtype=BF16)
    out, _ = bd.maxsim_attn_fwd(flat, flat, flat, cu_q=one, cu_k=one, max_q=3, max_k=3)
    assert torch.all(out == 0)
    for B, Lq, Lk in ((2, 0, 5), (2, 5, 0), (2, 0, 0)):
        q, k = e(B, Lq, 4, 64, dtype=BF16, device=DEV).fill_(1), e(B, Lk, 4, 64, dtype=BF16, device=DEV).fill_(1)
        out, lse = bd.maxsim_attn_fwd(q, k, k, with_lse=True)
        dq, dk, dv = bd.maxsim_attn_bwd(q, q, k, k, out, lse)
        assert torch.all(out == 0) and torch.all(lse == -math.inf) and torch.all(dq == 0) and torch.all(dk == 0) and torch.all(dv == 0)


@pytest.mark.parametrize("packed", [False, True])
def test_both_ways_of_making_a_call(bd, monkeypatch, packed):
    """The extension's calls and the general ones: the same results, views of any layout among them, and the same refusals."""
    s = state(bd, 3)
    taken = []
    for name in ("rope", "attn_fwd", "attn_bwd", "distill_fwd", "distill_bwd"):
        def count(*a, f=getattr(bd._fast, name), name=name):
            got = f(*a)
            taken.append((name, got is not None))
            return got
        monkeypatch.setattr(bd._fast, name, count)
    x, fused = s["x"], rand(2, 90, 9, 72, dtype=F16, seed=8)
    q, k, v, g = (fused[..., i:j, :64] for i, j in ((0, 4), (4, 6), (6, 8), (2, 6)))
    lens = dict(q_lens=s["how"]["q_lens"], k_lens=s["how"]["k_lens"])
    if packed:
        q, k, v, g = (t.flatten(0, 1) for t in (q, k, v, g))
        cu = torch.tensor([0, 100, 170], dtype=torch.int32, device=DEV)
        lens = dict(cu_q=cu, cu_k=cu, max_q=100, max_k=100)
    at = torch.randint(0, 1000, (2, 90), dtype=torch.int32, device=DEV)
    calls = [lambda **w: [bd.maxsim_rope(x, s["f"], positions=at, layout="interleaved", scale=1.25, inverse=True, **w)],
             lambda **w: [bd.maxsim_rope(x[:, :, 3:5], s["f"], offsets=s["off"], **w)],
             lambda **w: [t for t in bd.maxsim_attn_fwd(q, k, v, scale=0.3, window=(9, 3), sinks=1, **lens, **w) if t is not None],
             lambda **w: list(bd.maxsim_attn_fwd(q, k, v, with_lse=True, **lens, **w)),
             lambda **w: list(bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"], temperature=0.5, **w))]
    out, lse = bd.maxsim_attn_fwd(q, k, v, with_lse=True, **lens)
    _, stat = bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"])
    calls += [lambda **w: list(bd.maxsim_attn_bwd(g, q, k, v, out, lse, **lens, **w)),
              lambda **w: list(bd.maxsim_attn_bwd(g, q, k, v, out, lse.contiguous(), **lens, **w)),
              lambda **w: [bd.maxsim_distill_bwd(s["w"], s["z"], stat, s["index"], s["teacher"], **w)]]
    for call in calls:
        del taken[:]
        fast, general = call(), call(stream=torch.cuda.current_stream())
        assert taken and taken[-1][1], taken
        for a, b in zip(fast, general):
            assert a.shape == b.shape and a.dtype == b.dtype and a.stride() == b.stride() and torch.equal(a, b)
    for error, call in ((ValueError, lambda: bd.maxsim_rope(x, s["f"], layout="both")), (TypeError, lambda: bd.maxsim_rope(x, s["f"].float())),
                        (bd.MaxSimError, lambda: bd.maxsim_rope(x, s["f"], positions=at, offsets=s["off"])),
                        (bd.MaxSimError, lambda: bd.maxsim_attn_fwd(q, k, v, scale=-1.0, **lens)),
                        (bd.MaxSimError, lambda: bd.maxsim_attn_fwd(q, k, v, sinks=-1, **lens)),
                        (bd.MaxSimError, lambda: bd.maxsim_attn_fwd(q[..., 4:], k[..., 4:], v[..., 4:], **lens)),  # 8-byte aligned
                        (ValueError, lambda: bd.maxsim_attn_fwd(q, k, v[..., :56], **lens)),
                        (ValueError, lambda: bd.maxsim_attn_bwd(g, q, k, v, out, lse[..., :2], **lens)),
                        (bd.MaxSimError, lambda: bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"], temperature=0.0)),
                        (ValueError, lambda: bd.maxsim_distill_fwd(s["z"], s["index"], s["teacher"][:, :3]))):
        with pytest.raises(error):
            call()
