"""The embedding head and its training step as they are used together: the path
from hidden rows to MaxSim scores, gradients through the whole chain, captured
and replayed calls, other streams.  Run on an MI355X: pytest -m gpu."""
import pytest
import torch

import encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def randn(seed, *shape, scale=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def held(q, scale, br, bc):
    return q.double().cpu() * ref.spread(scale.double().cpu(), br, bc, q.shape)


@pytest.mark.parametrize("H", [256, 200])
def test_hidden_rows_to_scores(bd, H):
    """encode_tokens, then maxsim_fwd_varlen and maxsim_fwd_i8: scores against the 64-bit chain of the same operands."""
    Nq, Lq = 3, 32
    lens = [40, 7, 0, 129]
    cu = torch.tensor([0, 40, 47, 47, 176], dtype=torch.int32, device=DEV)
    hq, hd = randn(1, Nq, Lq, H, dtype=torch.bfloat16), randn(2, 176, H, dtype=torch.bfloat16)
    rq, rd = randn(3, Nq, Lq, H, dtype=torch.bfloat16), randn(4, 176, H, dtype=torch.bfloat16)
    gain, w = 1 + randn(5, H, scale=0.1), randn(6, 128, H, scale=H ** -0.5, dtype=torch.bfloat16)
    wq, ws, _, _ = bd.maxsim_quant_fp8(w, block_rows=128)

    def plain(x, r):
        _, _, y = ref.rmsnorm(x.cpu().reshape(-1, H), gain.cpu(), r.cpu().reshape(-1, H), 1e-6)
        cut = ref.blocks(y, 1, 128)
        s = cut.abs().amax(dim=(1, 3)) / 448
        y = (ref.round_e4m3(cut / s[:, None, :, None]) * s[:, None, :, None]).reshape(y.shape[0], -1)[:, :H]
        e = y @ held(wq, ws, 128, 128).t()
        return e / e.norm(dim=1, keepdim=True)

    pq, pd = plain(hq, rq).reshape(Nq, Lq, 128), plain(hd, rd)
    sim = torch.einsum("qid,td->qit", pq, pd)
    want = torch.stack([sim[:, :, int(cu[b]):int(cu[b + 1])].amax(2).sum(1) if lens[b] else torch.full((Nq,), -torch.inf).double()
                        for b in range(4)], 1)
    ok = torch.tensor(lens) > 0
    # bf16 rows: each of the 128 products of unit rows is off by 2 * 2^-9 of its magnitude at most, which sum to at
    # most 2^-8; codes that the fp32 norm rounds the other way are a few in a thousand of 2^-4 of a value
    Q, none = bd.encode_tokens(hq, gain, wq, ws, residual=rq, out_dtype=torch.bfloat16)
    D, _ = bd.encode_tokens(hd, gain, wq, ws, residual=rd, out_dtype=torch.bfloat16)
    assert none is None and Q.shape == (Nq, Lq, 128)
    s, _ = bd.maxsim_fwd_varlen(Q, D, cu, 129)
    assert torch.all(torch.isinf(s[:, 2])) and torch.all((s.cpu().double() - want).abs()[:, ok] <= 1.5 * 2.0 ** -8 * Lq)
    # int8 rows: half a step of at most 1 / 127 in each of 128 values on both sides: at most sqrt(128) / 127 / 2 each
    Q8, qs = bd.encode_tokens(hq, gain, wq, ws, residual=rq)
    D8, ds = bd.encode_tokens(hd, gain, wq, ws, residual=rd)
    assert Q8.dtype == torch.int8 and qs.shape == (Nq, Lq) and ds.shape == (176,)
    s8, _ = bd.maxsim_fwd_i8(Q8, qs, D8, ds, cu, 129)
    assert torch.all((s8.cpu().double() - want).abs()[:, ok] <= (2 * 128 ** 0.5 / 254 + 2.0 ** -8) * Lq)
    c, c8, i, v = bd.maxsim_two_stage_topk(Q8, qs, D8, ds, Q, D, cu, 129, 3, 2)
    # another kernel: 128 products and Lq maxima, each of magnitude at most 1 in all, added in another order
    assert torch.all((v[:, 0] - s.max(1).values).abs() <= 2 * (128 + Lq) * ref.U * Lq)


def test_rms_norm_autograd(bd):
    x, r, w = randn(1, 6, 5, 96), randn(2, 6, 5, 96), randn(3, 96)
    dy, ds = randn(4, 6, 5, 96), randn(5, 6, 5, 96)
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, s = bd.rms_norm(leaves[0], leaves[1], leaves[2])
    torch.autograd.backward([y, s], [dy, ds])
    plain = [t.double().requires_grad_() for t in (x, w, r)]
    h = plain[0] + plain[2]
    py = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * plain[1]
    torch.autograd.backward([py, h], [dy.double(), ds.double()])
    for a, b in zip(leaves, plain):
        assert torch.all((a.grad - b.grad).abs() <= 2.0 ** -17 * (1 + b.grad.abs()) * 8)
    # no residual, no gain, a frozen input, an expanded gradient, the same leaf twice
    a = x.clone().requires_grad_()
    bd.rms_norm(a).sum().backward()
    b = x.double().requires_grad_()
    (b * torch.rsqrt(b.square().mean(-1, keepdim=True) + 1e-6)).sum().backward()
    assert torch.all((a.grad - b.grad).abs() <= 2.0 ** -14)
    v = w.clone().requires_grad_()
    bd.rms_norm(x, v).backward(dy)
    assert v.grad is not None
    a = x.clone().requires_grad_()
    y, s = bd.rms_norm(a, w, a)
    y.backward(dy)
    b = x.double().requires_grad_()
    (2 * b * torch.rsqrt((2 * b).square().mean(-1, keepdim=True) + 1e-6) * w.double()).backward(dy.double())
    assert torch.all((a.grad - b.grad).abs() <= 2.0 ** -14 * (1 + b.grad.abs()))


@pytest.mark.parametrize("T,K,N", [(70, 200, 130), (300, 128, 128), (1, 64, 20)])
def test_linear_fp8_autograd(bd, T, K, N):
    """y, dx and dw against the 64-bit products of the operands that the quantiser makes."""
    x, w, dy = randn(1, T, K, dtype=torch.bfloat16), randn(2, N, K, dtype=torch.bfloat16), randn(3, T, N, dtype=torch.bfloat16)
    a, b = x.clone().requires_grad_(), w.float().requires_grad_()
    y = bd.linear_fp8(a, b)
    y.backward(dy)
    assert y.dtype == torch.bfloat16 and a.grad.dtype == torch.bfloat16 and b.grad.dtype == torch.float32
    q, s, qt, st = bd.maxsim_quant_fp8(x, transposed=True)
    wq, ws, wt, wst = bd.maxsim_quant_fp8(w.float(), block_rows=128, transposed=True)
    g, gs, gt, gst = bd.maxsim_quant_fp8(dy, transposed=True)
    for got, ops, rows in ((y, (q, s, wq, ws), 128), (a.grad, (g, gs, wt, wst), 128), (b.grad, (gt, gst, qt, st), 1)):
        want, size, largest = ref.gemm(*ops, rows)
        tol = ref.gemm_tolerance(want, size, largest, ops[0].shape[1], got.dtype)
        assert torch.all((got.detach().double().cpu() - want).abs() <= tol)
    frozen = bd.linear_fp8(x, b)
    frozen.backward(dy)
    only_x = x.clone().requires_grad_()
    bd.linear_fp8(only_x, w).sum().backward()   # an expanded gradient
    assert torch.isfinite(only_x.grad.float()).all()


def test_training_step(bd):
    """Norm, projection, norm, MaxSim, InfoNCE and AdamW: the gradients of the whole chain, along a direction, against
    central differences of the loss of the kernels' own forward with the argmax it chose and operands in 64 bits."""
    Nq, Lq, B, Ld, H = 4, 8, 4, 16, 256
    hq, hd = randn(1, Nq, Lq, H, dtype=torch.bfloat16), randn(2, B, Ld, H, dtype=torch.bfloat16)
    gain, w = 1 + randn(3, H, scale=0.1), randn(4, 128, H, scale=H ** -0.5)
    gain1 = torch.full((128,), 128 ** -0.5, device=DEV)
    params = [gain.clone().requires_grad_(), w.clone().requires_grad_()]

    def loss_of(gain, w):
        rows = [bd.rms_norm(bd.linear_fp8(bd.rms_norm(h, gain), w), gain1) for h in (hq, hd)]
        scores = bd.maxsim(rows[0], rows[1])
        return torch.nn.functional.cross_entropy(scores / 0.5, torch.arange(Nq, device=DEV)), rows

    loss, rows = loss_of(*params)
    loss.backward()
    _, arg = bd.maxsim_fwd(*[r.detach() for r in rows])
    arg = arg.cpu().long()

    def plain(gain, w):
        out = []
        for h in (hq, hd):
            x = h.double().cpu()
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain
            e = x @ w.t()
            out.append(e * torch.rsqrt(e.square().mean(-1, keepdim=True) + 1e-6) * 128 ** -0.5)
        picked = out[1][torch.arange(B)[None, :, None], arg]          # [Nq, B, Lq, 128]
        scores = (out[0][:, None] * picked).sum((2, 3))
        return torch.nn.functional.cross_entropy(scores / 0.5, torch.arange(Nq))

    leaves = [gain.double().cpu().requires_grad_(), w.double().cpu().requires_grad_()]
    plain(*leaves).backward()
    # the plain gradient against differences
    d = [torch.randn(t.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(9)) for t in leaves]
    step = 1e-5
    with torch.no_grad():
        diff = (plain(*[t + step * u for t, u in zip(leaves, d)]) - plain(*[t - step * u for t, u in zip(leaves, d)])) / (2 * step)
    along = sum((t.grad * u).sum() for t, u in zip(leaves, d))
    assert abs(diff - along) <= 1e-6 * (1 + abs(along))
    # the chain's: values in 8 bits are off by 2^-4 / sqrt(3) or so of themselves at random, in three products in turn
    for got, want in zip(params, leaves):
        err = float((got.grad.double().cpu() - want.grad).norm() / want.grad.norm())
        assert err <= 3 * 2.0 ** -4, err
    # and the optimiser takes them
    tab = bd.AdamWTensors.zeros(params)
    before = [p.detach().clone() for p in params]
    bd.maxsim_adamw(tab, [p.grad for p in params], 1, lr=1e-3, weight_decay=0.0)
    for p, q in zip(params, before):
        moved = (p.detach() - q).abs()
        assert torch.all(moved <= 1e-3 * (1 + 1e-4) + 4 * ref.U) and torch.any(moved > 5e-4)


def chain(bd, x, res, gain, wq, ws, dy):
    q, s, h, r = bd.maxsim_rmsnorm_fwd(x, gain, residual=res, out_dtype=torch.float8_e4m3fn, with_rstd=True)
    c = bd.maxsim_gemm_fp8(q, s, wq, ws, out_dtype=torch.float32)   # splits K
    few = bd.maxsim_gemm_fp8(q[:20], s[:20], wq, ws)
    dx, dw = bd.maxsim_rmsnorm_bwd(dy, h, r, gain)
    t = bd.maxsim_quant_fp8(dy, transposed=True)
    return (q, s, h, r, c, few, dx, dw) + t


def test_captured_and_replayed(bd):
    """The operators in a graph, replayed on new inputs with eager work between: every replay equals the eager call."""
    R, H, N = 150, 4096, 128
    x, res, dy = (torch.empty(R, H, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    gain = 1 + randn(5, H, scale=0.1)
    wq, ws, _, _ = bd.maxsim_quant_fp8(randn(6, N, H), block_rows=128)
    for t, i in ((x, 1), (res, 2), (dy, 3)):
        t.copy_(randn(i, R, H))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(bd, x, res, gain, wq, ws, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(bd, x, res, gain, wq, ws, dy)
    for k in range(4):
        for t, i in ((x, 1), (res, 2), (dy, 3)):
            t.copy_(randn(10 * k + i, R, H))
        graph.replay()
        torch.cuda.synchronize()
        want = chain(bd, x, res, gain, wq, ws, dy)
        for a, b in zip(out, want):
            assert torch.equal(a.float(), b.float()), k


def test_two_streams_at_once(bd):
    """The same calls on two streams, with stream= and with the current stream, give what one stream gives."""
    R, H, N = 300, 2048, 128
    gain = 1 + randn(5, H, scale=0.1)
    wq, ws, _, _ = bd.maxsim_quant_fp8(randn(6, N, H), block_rows=128)
    ins = [[randn(7 * k + i, R, H, dtype=torch.bfloat16) for i in range(3)] for k in range(2)]
    want = [chain(bd, *a[:2], gain, wq, ws, a[2]) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(chain(bd, *ins[k][:2], gain, wq, ws, ins[k][2]))
    for s in streams:
        s.synchronize()
    for k in range(2):
        for run in got[k]:
            for a, b in zip(run, want[k]):
                assert torch.equal(a.float(), b.float())
    q, s, _, _ = bd.maxsim_rmsnorm_fwd(ins[0][0], gain, out_dtype=torch.float8_e4m3fn, stream=streams[0])
    c = bd.maxsim_gemm_fp8(q, s, wq, ws, stream=streams[0])
    streams[0].synchronize()
    q2, s2, _, _ = bd.maxsim_rmsnorm_fwd(ins[0][0], gain, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(c, bd.maxsim_gemm_fp8(q2, s2, wq, ws))


@pytest.mark.parametrize("H", [256, 129])
def test_both_ways_through_the_binding(bd, H):
    """The usual calls go through the extension, all others through ctypes: the same results, and the extension leaves
    alone what it does not handle."""
    here = torch.cuda.current_stream()
    same = lambda a, b: all((x is None and y is None) or (x.shape == y.shape and x.dtype == y.dtype  # noqa: E731
                                                          and torch.equal(x.float(), y.float())) for x, y in zip(a, b))
    x, r, w = randn(1, 5, 7, H), randn(2, 5, 7, H), randn(3, H)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        for out in (None, torch.float32, torch.int8, torch.float8_e4m3fn):
            for res in (None, r.to(dt)):
                a = bd.maxsim_rmsnorm_fwd(x.to(dt), w, residual=res, out_dtype=out, with_rstd=True)
                b = bd.maxsim_rmsnorm_fwd(x.to(dt), w, residual=res, out_dtype=out, with_rstd=True, stream=here)
                assert same(a, b)
        h, rstd = x.to(dt), b[3]
        for dsum in (None, r.to(dt)):
            for with_dweight in (True, False):
                assert same(bd.maxsim_rmsnorm_bwd(r.to(dt), h, rstd, w, dsum, with_dweight),
                            bd.maxsim_rmsnorm_bwd(r.to(dt), h, rstd, w, dsum, with_dweight, stream=here))
        m = randn(4, 160, H, dtype=dt)
        for br in (1, 128):
            for rows, both in ((True, False), (True, True), (False, True)):
                assert same(bd.maxsim_quant_fp8(m, br, rows, both), bd.maxsim_quant_fp8(m, br, rows, both, stream=here))
    q, s, _, _ = bd.maxsim_quant_fp8(randn(4, 160, H))
    b, bs, _, _ = bd.maxsim_quant_fp8(randn(5, 100, H), 128)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        assert same([bd.maxsim_gemm_fp8(q, s, b, bs, dt)], [bd.maxsim_gemm_fp8(q, s, b, bs, dt, stream=here)])
        assert same([bd.maxsim_gemm_fp8(q, s, q, s, dt)], [bd.maxsim_gemm_fp8(q, s, q, s, dt, stream=here)])
    tabs = [bd.AdamWTensors.zeros([randn(6, 70), randn(7, 300)], torch.float8_e4m3fn) for _ in range(2)]
    g = [randn(8, 70), randn(9, 300)]
    before = tabs[0]._table.copy()
    bd.maxsim_adamw(tabs[0], g, 1)
    bd.maxsim_adamw(tabs[1], g, 1, stream=here)
    assert (tabs[0]._table == before).all()
    for f in ("params", "m", "v", "m_scales", "v_scales"):
        assert same(getattr(tabs[0], f), getattr(tabs[1], f)), f
    # not for the extension: None, and no launch
    t = randn(1, 6, H)
    assert bd._fast.rmsnorm_fwd(t[:, ::2], None, 1e-6, None, None, False) is None
    assert bd._fast.rmsnorm_fwd(t.cpu(), None, 1e-6, None, None, False) is None
    assert bd._fast.rmsnorm_fwd(t, t, 1e-6, None, None, False) is None
    assert bd._fast.rmsnorm_fwd("x", None, 1e-6, None, None, False) is None
    assert bd._fast.rmsnorm_fwd(t) is None
    assert bd._fast.quant_fp8(t, 64, True, False) is None and bd._fast.quant_fp8(t.double(), 1, True, False) is None
    assert bd._fast.gemm_fp8(q, s, b, bs[:0], torch.float32) is None
    assert bd._fast.gemm_fp8(q, s, b, bs, torch.int8) is None
    assert bd._fast.rmsnorm_bwd(t, t, t, None, None, True) is None
    assert bd._fast.adamw(tabs[0]._address, 2, 0, 2, 4, g[:1], 1e-3, .9, .99, 1e-8, 0., 1) is None


def test_autograd_corners(bd):
    """No tokens, views that are not contiguous, a leaf used twice, a second derivative (refused)."""
    w = randn(1, 130, 64).requires_grad_()
    x = torch.zeros(0, 64, device=DEV, requires_grad=True)
    y = bd.linear_fp8(x, w)
    y.sum().backward()
    assert y.shape == (0, 130) and x.grad.shape == (0, 64) and torch.all(w.grad == 0)
    wide = randn(2, 64, 50)
    a, b = wide.t().clone().requires_grad_(), wide.clone().requires_grad_()
    v = randn(3, 64, 130)
    bd.linear_fp8(a, v.t()).square().sum().backward()
    bd.linear_fp8(b.t(), v.t().contiguous()).square().sum().backward()
    assert torch.equal(a.grad, b.grad.t())
    n = bd.rms_norm(b.detach().t())
    assert torch.equal(n, bd.rms_norm(b.detach().t().contiguous()))
    both = randn(4, 40, 64).requires_grad_()
    one, two = both.detach().clone().requires_grad_(), both.detach().clone().requires_grad_()
    (bd.linear_fp8(both, w.detach()).sum() + 2 * bd.linear_fp8(both, w.detach()).sum()).backward()
    bd.linear_fp8(one, w.detach()).sum().backward()
    (2 * bd.linear_fp8(two, w.detach()).sum()).backward()
    assert torch.allclose(both.grad, one.grad + two.grad, rtol=4 * ref.U, atol=0)
    x = randn(5, 4, 64).requires_grad_()
    g, = torch.autograd.grad(bd.rms_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
