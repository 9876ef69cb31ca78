"""The AdamW step over many tensors against the 64-bit formula, states in fp32
and in 8 bits.  Run on an MI355X: pytest -m gpu.

Tolerances: a moment is two products and a sum in fp32 (4 u of the magnitudes,
the rounded factors among them); the update's chain of seven operations (16 u
of itself) is added to p with one rounding."""
import pytest
import torch

import encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05)
SIZES = [1, 7, 128, 129, 2048, 2049, 5000, 1, 100, 70000]


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def state(seed, sizes, dtype, grad_dtype, off=0):
    """Tensors that start `off` elements into their memory."""
    g = torch.Generator().manual_seed(seed)

    def make(scale, dt, positive=False):
        out = []
        for n in sizes:
            t = torch.randn(n + off, generator=g) * scale
            out.append((t.abs() if positive else t).to(dt).to(DEV)[off:])
        return out

    return dict(p=make(0.1, dtype), g=make(1e-3, grad_dtype), m=make(1e-3, torch.float32),
                v=make(1e-6, torch.float32, True), w=make(0.1, torch.float32))


def want_of(p, g, m, v, t):
    return ref.adamw(p.cpu(), g.cpu(), m.cpu(), v.cpu(), t, *HYPER.values())


def check_params(got, want, before, dtype, where):
    move = (want - before.double()).abs()
    tol = ref.half_step(dtype) * want.abs() * (1 + 1e-3) + 16 * ref.U * move + 4 * ref.U * before.double().abs()
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert torch.all((got.double().cpu() - want).abs() <= tol), where


@pytest.mark.parametrize("dtype,grad", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                        (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                        (torch.float16, torch.float16), (torch.bfloat16, torch.float32)], ids=str)
@pytest.mark.parametrize("off", [0, 1])
def test_fp32_states(bd, dtype, grad, off):
    s = state(1, SIZES, dtype, grad, off)
    for masters in (False, True):
        if masters and dtype == torch.float32:
            continue
        p, m, v = [t.clone() for t in s["p"]], [t.clone() for t in s["m"]], [t.clone() for t in s["v"]]
        w = [t.clone() for t in s["w"]] if masters else None
        if off:  # keep the odd alignment
            p, m, v = s["p"], s["m"], s["v"]
        before = [(t.clone(), a.clone(), b.clone()) for t, a, b in zip(w or p, m, v)]
        bd.maxsim_adamw(bd.AdamWTensors(p, m, v, masters=w), s["g"], 7, **HYPER)
        for i in range(len(SIZES)):
            bp, bm, bv = before[i]
            wp, wm, wv = want_of(bp, s["g"][i], bm, bv, 7)
            check_params(p[i], wp, bp.cpu(), dtype, i)
            if masters:
                check_params(w[i], wp, bp.cpu(), torch.float32, i)
                assert torch.equal(p[i], w[i].to(dtype))
            g = s["g"][i].double().cpu()
            assert torch.all((m[i].double().cpu() - wm).abs() <= 4 * ref.U * (bm.double().cpu().abs() + g.abs()))
            assert torch.all((v[i].double().cpu() - wv).abs() <= 6 * ref.U * (bv.double().cpu() + g * g))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_8_bit_states(bd, dtype):
    """Three steps; each checked against the formula from the states the kernel left before it."""
    s = state(2, SIZES, dtype, torch.float32)
    tab = bd.AdamWTensors.zeros(s["p"], torch.float8_e4m3fn)
    flat = lambda q, c: q.double().cpu() * c.double().cpu().repeat_interleave(128)[:q.numel()]  # noqa: E731
    for t in (1, 2, 3):
        held = tab.masters or tab.params
        before = [(x.clone(), flat(m, ms), flat(v, vs) ** 2)
                  for x, m, ms, v, vs in zip(held, tab.m, tab.m_scales, tab.v, tab.v_scales)]
        grads = [g * t for g in s["g"]]
        bd.maxsim_adamw(tab, grads, t, **HYPER)
        for i, (bp, bm, bv) in enumerate(before):
            wp, wm, wv = want_of(bp, grads[i], bm, bv, t)
            check_params(held[i], wp, bp.cpu(), torch.float32, (t, i))
            if tab.masters:
                assert torch.equal(tab.params[i], held[i].to(dtype))
            ref.check_held(tab.m[i][None], tab.m_scales[i][None], wm[None], 1, 128, "e4m3", 2.0 ** -21, "m")
            root = wv.sqrt()
            q = tab.v[i].double().cpu()
            # a root that is not 0 is at least the smallest code, where the nearest may be 0
            sc = tab.v_scales[i].double().cpu().repeat_interleave(128)[:q.numel()]
            raised = (q == 2.0 ** -9) & (root / sc < 2.0 ** -9)
            ref.check_held(torch.where(raised, root / sc, q)[None], tab.v_scales[i][None], root[None], 1, 128, "e4m3",
                           2.0 ** -21, "v")
            assert torch.all(q[(root > 0) & (sc != 1)] > 0)


def test_roots_are_never_lost(bd):
    """One large gradient in a block of small ones: their roots stay above 0, and the next step is bounded."""
    p = [torch.zeros(128, device=DEV)]
    tab = bd.AdamWTensors.zeros(p, torch.float8_e4m3fn)
    g = torch.full((128,), 1e-7, device=DEV)
    g[5] = 1.0
    bd.maxsim_adamw(tab, [g], 1, lr=1e-3, beta1=0.9, beta2=0.999, eps=0.0, weight_decay=0.0)
    assert torch.all(tab.v[0].float() > 0)
    bd.maxsim_adamw(tab, [torch.zeros_like(g)], 2, lr=1e-3, beta1=0.9, beta2=0.999, eps=0.0, weight_decay=0.0)
    assert torch.isfinite(tab.params[0]).all()


def test_many_tensors(bd):
    """More tensors than one launch's table holds, empty ones among them."""
    sizes = [(i * 37) % 300 for i in range(171)]
    s = state(3, sizes, torch.float32, torch.float32)
    before = [(a.clone(), b.clone(), c.clone()) for a, b, c in zip(s["p"], s["m"], s["v"])]
    bd.maxsim_adamw(bd.AdamWTensors(s["p"], s["m"], s["v"]), s["g"], 2, **HYPER)
    for i in range(len(sizes)):
        wp, _, _ = want_of(before[i][0], s["g"][i], *before[i][1:], 2)
        check_params(s["p"][i], wp, before[i][0].cpu(), torch.float32, i)


@pytest.mark.parametrize("state_dtype", [torch.float32, torch.float8_e4m3fn], ids=str)
def test_neighbours_are_left(bd, state_dtype):
    """The values on both sides of a tensor stay as they were."""
    n = 300
    big = [torch.full((n + 64,), 7.0, device=DEV) for _ in range(3)] + [torch.full((n + 64,), 2.0, device=DEV)]
    view = lambda t: t[32:32 + n]  # noqa: E731
    if state_dtype == torch.float32:
        tab = bd.AdamWTensors([view(big[0])], [view(big[1])], [view(big[2])])
    else:
        big[1], big[2] = big[1].to(state_dtype), big[2].to(state_dtype)
        sc = [torch.full((5,), 7.0, device=DEV) for _ in range(2)]
        tab = bd.AdamWTensors([view(big[0])], [view(big[1])], [view(big[2])], [sc[0][1:4]], [sc[1][1:4]])
    bd.maxsim_adamw(tab, [view(big[3])], 1, **HYPER)
    assert torch.all(big[3] == 2)
    for t in big[:3]:
        t = t.float()
        assert torch.all(t[:32] == 7) and torch.all(t[32 + n:] == 7) and torch.any(t[32:32 + n] != 7)
    if state_dtype != torch.float32:
        for c in sc:
            assert c[0] == 7 and c[4] == 7 and torch.all(c[1:4] != 7)


def test_step_on_the_device_and_replay(bd):
    """A captured step counts its replays through step_dev and equals eager steps, 8-bit states included."""
    for state_dtype in (torch.float32, torch.float8_e4m3fn):
        s = state(4, [5000, 33], torch.float32, torch.float32)
        eager = bd.AdamWTensors.zeros([p.clone() for p in s["p"]], state_dtype)
        replay = bd.AdamWTensors.zeros([p.clone() for p in s["p"]], state_dtype)
        grads = [torch.zeros_like(g) for g in s["g"]]
        count = torch.zeros(1, dtype=torch.int32, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            bd.maxsim_adamw(bd.AdamWTensors.zeros([torch.zeros(5, device=DEV)]), [torch.zeros(5, device=DEV)], 1)
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            count += 1
            bd.maxsim_adamw(replay, grads, 0, step_dev=count, **HYPER)
        for t in range(1, 5):
            now = [g * t for g in s["g"]]
            for a, b in zip(grads, now):
                a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            bd.maxsim_adamw(eager, now, t, **HYPER)
            assert int(count) == t
            for a, b in zip(eager.params, replay.params):
                # the same kernel; the host's and the device's expm1 may differ in the last place
                assert torch.all((a - b).abs() <= 4 * ref.U * (a.abs() + HYPER["lr"] * t))


def test_binding_refusals(bd):
    s = state(1, [5, 6], torch.float32, torch.float32)
    tab = bd.AdamWTensors(s["p"], s["m"], s["v"])
    for bad in (s["g"][:1], [s["g"][0], s["g"][1].bfloat16()], [s["g"][0], s["g"][0]], [t.cpu() for t in s["g"]]):
        with pytest.raises(ValueError):
            bd.maxsim_adamw(tab, bad, 1)
    with pytest.raises(TypeError):
        bd.maxsim_adamw(tab, [g.int() for g in s["g"]], 1)
    with pytest.raises(bd.MaxSimError):
        bd.maxsim_adamw(tab, s["g"], 0)
    with pytest.raises(TypeError):
        bd.maxsim_adamw(tab, s["g"], 0, step_dev=torch.zeros(1, device=DEV))


@pytest.mark.parametrize("device_step", [False, True])
def test_parameters_of_autograd(bd, device_step):
    """A parameter whose memory was replaced is refused, and a graph that saved one before the step refuses its
    backward: both ways of making the call."""
    w = torch.nn.Parameter(torch.ones(200, device=DEV))
    tab = bd.AdamWTensors.zeros([w])
    step = dict(step_dev=torch.ones(1, dtype=torch.int32, device=DEV)) if device_step else {}
    loss = (w * w).sum()
    bd.maxsim_adamw(tab, [torch.ones(200, device=DEV)], 1, **step)
    assert torch.all(w < 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        plain = torch.ones(200, device=DEV)
    bd.maxsim_adamw(bd.AdamWTensors.zeros([plain]), [torch.ones(200, device=DEV)], 1, **step)
    assert torch.equal(plain, w.detach())
    was = w.data
    w.data = was.clone()
    with pytest.raises(ValueError, match="moved"):
        bd.maxsim_adamw(tab, [torch.ones(200, device=DEV)], 2, **step)
    assert torch.equal(was, w.data)
