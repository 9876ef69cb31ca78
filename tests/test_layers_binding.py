"""The binding of the attention layer's operators and of the distillation loss on a host without a GPU: what it refuses
before any device work, rotary frequencies, and the references' bounds, which have to see a planted mistake."""
import math

import numpy as np
import pytest
import torch

import layers_ref as ref
from late_interaction_retrieval_amd import binding as bd

BF16 = torch.bfloat16


def meta(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_host_tensors_are_refused():
    x, i = torch.zeros(2, 3, 4, 64, dtype=BF16), torch.zeros(4, 2, dtype=torch.int32)
    s = torch.zeros(4, 8)
    for call in (lambda: bd.maxsim_rope(x, torch.zeros(32)), lambda: bd.maxsim_attn_fwd(x, x, x),
                 lambda: bd.maxsim_attn_bwd(x, x, x, x, x, s), lambda: bd.maxsim_distill_fwd(s, i, s[:, :2]),
                 lambda: bd.maxsim_distill_bwd(s[:, 0], s, s[:, :2], i, s[:, :2]), lambda: bd.attention(x, x, x),
                 lambda: bd.rope(x, torch.zeros(32)), lambda: bd.distill_loss(s, i, s[:, :2])):
        with pytest.raises(ValueError, match="must be on the device"):
            call()


def rope(x, f=None, positions=None, offsets=None, layout="half", scale=1.0, inverse=False, out=None):
    return bd._rope.__wrapped__(x, meta(32, dtype=torch.float64) if f is None else f, positions, offsets, layout, scale, inverse, out)


@pytest.mark.parametrize("error,kw", [
    (ValueError, dict(x=meta(3, 64))), (ValueError, dict(layout="both")), (TypeError, dict(x=meta(2, 3, 4, 64, dtype=torch.int32))),
    (TypeError, dict(f=meta(32, dtype=torch.float32))), (ValueError, dict(positions=meta(5, dtype=torch.int32))),
    (TypeError, dict(positions=meta(2, 3, dtype=torch.int64))), (ValueError, dict(offsets=meta(3, dtype=torch.int32))),
    (ValueError, dict(x=meta(2, 3, 4, 128)[..., ::2])), (ValueError, dict(out=meta(2, 3, 4, 63))),
    (TypeError, dict(out=meta(2, 3, 4, 64, dtype=torch.float16))), (ValueError, dict(out=torch.zeros(2, 3, 4, 64, dtype=BF16))),
    (ValueError, dict(x=meta(1, (1 << 32) + 5, 1, 64))),
], ids=str)
def test_rope_arguments(error, kw):
    kw = dict(kw)
    with pytest.raises(error):
        rope(kw.pop("x", meta(2, 3, 4, 64)), **kw)


def attn(q=None, k=None, v=None, out=None, **kw):
    a = dict(scale=None, window=(-1, -1), sinks=0, q_lens=None, k_lens=None, cu_q=None, cu_k=None, max_q=None, max_k=None)
    a.update(kw)
    q, k = meta(2, 3, 4, 64) if q is None else q, meta(2, 9, 2, 64) if k is None else k
    return bd._attn(q, k, k if v is None else v, out, *a.values())


@pytest.mark.parametrize("error,kw", [
    (ValueError, dict(q=meta(3, 4, 64))), (ValueError, dict(cu_q=meta(3, dtype=torch.int32))), (ValueError, dict(k=meta(3, 9, 2, 64))),
    (ValueError, dict(k=meta(2, 9, 2, 32))), (ValueError, dict(v=meta(2, 8, 2, 64))), (TypeError, dict(k=meta(2, 9, 2, 64, dtype=torch.float16))),
    (TypeError, dict(q=meta(2, 3, 4, 64, dtype=torch.float32))), (ValueError, dict(out=meta(2, 3, 4, 32))),
    (ValueError, dict(q_lens=meta(3, dtype=torch.int32))), (TypeError, dict(k_lens=meta(2, dtype=torch.int64))),
    (ValueError, dict(q=meta(7, 4, 64), cu_q=meta(3, dtype=torch.int32))),  # no max_q
    (ValueError, dict(q=meta(7, 4, 64), cu_q=meta(3, dtype=torch.int32), max_q=5, q_lens=meta(2, dtype=torch.int32))),
    (ValueError, dict(q=meta(7, 4, 64), cu_q=meta(4, dtype=torch.int32), max_q=5)),  # three sequences for two
    (ValueError, dict(window=(1 << 32, 0))), (ValueError, dict(sinks=1 << 31)), (ValueError, dict(q=meta(2, 3, 4, 128)[..., ::2])),
], ids=str)
def test_attention_arguments(error, kw):
    with pytest.raises(error):
        attn(**kw)


def test_attention_struct():
    a = attn(window=(5, 0), sinks=2)
    assert (a.B, a.max_q, a.max_k, a.Hq, a.Hk, a.D) == (2, 3, 9, 4, 2, 64) and (a.left, a.right, a.sinks) == (5, 0, 2)
    assert (a.q.batch, a.q.token, a.q.head) == (768, 256, 64) and abs(a.scale - 0.125) < 1e-9
    moved = attn(q=meta(2, 4, 3, 64).transpose(1, 2))
    assert (moved.q.batch, moved.q.token, moved.q.head) == (768, 64, 192)
    one = attn(q=meta(1, 1, 1, 64), k=meta(1, 1, 1, 64).as_strided((1, 1, 1, 64), (0, 0, 0, 1)))
    assert (one.k.batch, one.k.token, one.k.head) == (0, 64, 64)


def test_lse_of_both_kinds():
    q = torch.zeros(2, 5, 3, 64)
    state = torch.zeros(2, 5, 3, 33)
    assert bd._lse_step(state[..., 0], q) == 33 and bd._lse_step(state[..., 0].contiguous(), q) == 1
    assert bd._lse_step(torch.zeros(5, 1, 33)[..., 0], q[0, :, :1]) == 33
    for bad in (state[..., :3], torch.zeros(2, 5, 3, 8)[..., 0], torch.zeros(2, 5, 3).transpose(0, 1), state[:, :4, :, 0],
                torch.zeros(2, 6, 3, 33)[:, :5, :, 0], state[..., 0].double(), state[..., 1]):
        with pytest.raises(ValueError):
            bd._lse_step(bad, q)


def test_distill_arguments():
    raw = bd._distill_fwd.__wrapped__
    z, i, t = meta(4, 9, dtype=torch.float32), meta(4, 2, dtype=torch.int32), meta(4, 2, dtype=torch.float32)
    for bad in ((z[0], i, t), (z, i[0], t), (z, i, t[:, :1]), (z, meta(3, 2, dtype=torch.int32), t), (z.t(), i, t)):
        with pytest.raises(ValueError):
            raw(*bad, 1.0, None, None, None)
    for bad in ((z, i.long(), t), (z, i, t.double()), (z.long(), i, t)):
        with pytest.raises(TypeError):
            raw(*bad, 1.0, None, None, None)


def test_rope_frequencies():
    f, scale = bd.rope_frequencies(64, device="cpu")
    i = np.arange(32)
    assert scale == 1.0 and f.dtype == torch.float64
    assert np.allclose(f.numpy(), 10000.0 ** (-i / 32), rtol=1e-14)
    g, scale = bd.rope_frequencies(64, stretch=4.0, kind="linear", device="cpu")
    assert scale == 1.0 and np.allclose(g.numpy(), f.numpy() / 4, rtol=1e-14)
    g, scale = bd.rope_frequencies(64, stretch=4.0, kind="base", device="cpu")  # the slowest is divided, the fastest stays
    assert scale == 1.0 and abs(g[0] - 1) < 1e-14 and abs(g[-1] / f[-1] - 0.25) < 1e-12
    g, scale = bd.rope_frequencies(64, stretch=4.0, kind="parts", length=4096, device="cpu")
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert abs(scale - (1 + 0.1 * math.log(4))) < 1e-12
    assert np.allclose(g.numpy()[turns > 32], f.numpy()[turns > 32], rtol=1e-14)
    assert np.allclose(g.numpy()[turns < 1], f.numpy()[turns < 1] / 4, rtol=1e-14)
    between = (turns < 32) & (turns > 1)
    assert between.any() and np.all(g.numpy()[between] < f.numpy()[between]) and np.all(g.numpy()[between] > f.numpy()[between] / 4)
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=8, kind="other"), dict(rotary=8, stretch=0.5), dict(rotary=8, base=-1.0)):
        with pytest.raises(ValueError):
            bd.rope_frequencies(device="cpu", **bad)


# ---------------------------------------------------------------- the references' bounds


def inputs(L=90, H=2, D=32, dtype=BF16):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(L, H, D, generator=g).to(dtype) for _ in range(4)]


def plain(q, k, v, g, window, sinks):
    """Attention and its gradients in fp32, rounded once, one head for each."""
    T = q.dtype
    q, k, v = (t.float().requires_grad_() for t in (q, k, v))
    vis = ref.seen(q.shape[0], k.shape[0], window, sinks)
    o = torch.stack([torch.softmax((q[:, h] @ k[:, h].t() * q.shape[-1] ** -0.5).masked_fill(~vis, -math.inf), 1) @ v[:, h]
                     for h in range(q.shape[1])], 1)
    return {"out": o.detach().to(T), **{n: t.to(T) for n, t in zip(("dq", "dk", "dv"), torch.autograd.grad(o, (q, k, v), g.float()))}}


@pytest.mark.parametrize("dtype", [torch.float16, BF16], ids=str)
def test_a_right_result_is_within_bounds_and_a_window_off_by_one_is_not(dtype):
    q, k, v, g = inputs(dtype=dtype)
    want = ref.attention(q, k, v, [(0, 90, 0, 90)], 32 ** -0.5, (20, 0), 2, g)
    good = plain(q, k, v, g, (20, 0), 2)
    for n in good:
        ref.check(good[n], want[n], n)
    for window, sinks in (((21, 0), 2), ((19, 0), 2), ((20, 1), 2), ((20, 0), 3), ((20, 0), 1)):
        wrong = plain(q, k, v, g, window, sinks)
        for n in wrong:
            with pytest.raises(AssertionError):
                ref.check(wrong[n], want[n], n)


def test_a_wrong_angle_or_pair_is_seen():
    x = torch.randn(9, 2, 16, generator=torch.Generator().manual_seed(2))
    f, _ = bd.rope_frequencies(12, device="cpu")
    at = torch.arange(9)
    want = ref.rope(x, f, at, "half", 1.0)
    ref.check(want[0].float(), want, "itself")
    for wrong in (ref.rope(x, f, at + 1, "half", 1.0), ref.rope(x, f, at, "interleaved", 1.0), ref.rope(x, f, at, "half", 1.0, True),
                  ref.rope(x, f * (1 + 1e-5), at, "half", 1.0)):
        with pytest.raises(AssertionError):
            ref.check(wrong[0].float(), want, "wrong")


def test_the_loss_is_the_formulas():
    g = torch.Generator().manual_seed(3)
    z = torch.randn(5, 30, generator=g).requires_grad_()
    index = torch.stack([torch.randperm(30, generator=g)[:4] for _ in range(5)]).to(torch.int32)
    t, dloss = torch.randn(5, 4, generator=g), torch.rand(5, generator=g)
    want = ref.distill(z.detach(), index, t, 2.0, dloss)
    target = torch.softmax(t / 2, 1)
    loss = 4 * (target * (target.log() - torch.log_softmax(z / 2, 1).gather(1, index.long()))).sum(1)
    ref.check(loss.detach(), want["loss"], "loss")
    ref.check(torch.autograd.grad(loss, z, dloss)[0], want["dscores"], "dscores")
    ref_wrong = ref.distill(z.detach(), index, t, 2.001, dloss)
    with pytest.raises(AssertionError):
        ref.check(ref_wrong["loss"][0], want["loss"], "loss")
