"""The binding of the embedding head's operators on a host without a GPU: which way a call takes, and what it refuses
before any device work."""
import copy
import io
import os
import subprocess
import sys

import pytest
import torch

from late_interaction_retrieval_amd import binding as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def step(monkeypatch):
    """A table of host tensors, and the C entry point replaced by one that counts its calls."""
    calls = []
    tab = bd.AdamWTensors.zeros([torch.zeros(5)])

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def maxsim_adamw(self, *args):
            calls.append(args)
            return bd.MAXSIM_OK

    real = bd._lib
    monkeypatch.setattr(bd, "_lib", Lib())
    return tab, calls


@pytest.mark.parametrize("status", range(1, 8))
def test_a_step_that_failed_is_not_made_again(step, monkeypatch, status):
    """The extension's call may have launched a part of the step: its status is raised, and no second call follows."""
    tab, calls = step
    monkeypatch.setattr(bd._fast, "adamw", lambda *a: status)
    with pytest.raises(bd.MaxSimError) as e:
        bd.maxsim_adamw(tab, [torch.zeros(5)], 1)
    assert e.value.status == status and not calls


def test_a_step_that_was_made_is_not_made_again(step, monkeypatch):
    tab, calls = step
    monkeypatch.setattr(bd._fast, "adamw", lambda *a: bd.MAXSIM_OK)
    assert bd.maxsim_adamw(tab, [torch.zeros(5)], 1) is None and not calls


def test_a_step_that_the_extension_leaves_alone_goes_the_general_way(step, monkeypatch):
    tab, calls = step
    monkeypatch.setattr(bd._fast, "adamw", lambda *a: None)
    with pytest.raises(ValueError, match="must be on the device"):  # host tensors
        bd.maxsim_adamw(tab, [torch.zeros(5)], 1)


@pytest.fixture
def norm_on_host(monkeypatch):
    """The norm's two calls by plain torch on the host; what the backward is given is kept."""
    seen = []

    def fwd(x, weight=None, eps=1e-6, residual=None, with_rstd=False):
        h = x if residual is None else x + residual
        rstd = torch.rsqrt(h.square().mean(-1) + eps)
        return h * rstd[..., None] * (1 if weight is None else weight.reshape(-1)), None, None if residual is None else h, rstd

    def bwd(dy, h, rstd, weight=None, dsum=None, with_dweight=True):
        seen.append((dy, dsum))
        g, xh = dy * (1 if weight is None else weight.reshape(-1)), h * rstd[..., None]
        dx = rstd[..., None] * (g - xh * (g * xh).mean(-1, keepdim=True)) + (0 if dsum is None else dsum)
        return dx, (dy * xh).flatten(0, -2).sum(0) if with_dweight else None

    monkeypatch.setattr(bd, "maxsim_rmsnorm_fwd", fwd)
    monkeypatch.setattr(bd, "maxsim_rmsnorm_bwd", bwd)
    return seen


@pytest.mark.parametrize("use_y,use_sum", [(True, False), (False, True), (True, True)])
def test_outputs_of_the_norm_that_nothing_uses(norm_on_host, use_y, use_sum):
    """An output without a gradient reaches the backward as none, not as zeros; the gradients are the formula's."""
    g = torch.Generator().manual_seed(1)
    x, w, r = (torch.randn(s, generator=g, dtype=torch.float64).requires_grad_() for s in ((3, 8), (8,), (3, 8)))
    dy, ds = (torch.randn(3, 8, generator=g, dtype=torch.float64) for _ in range(2))

    def loss(y, h):
        if use_y and use_sum:
            return (y * dy).sum() + (h * ds).sum()
        return (y * dy if use_y else h * ds).sum()

    loss(*bd.rms_norm(x, w, residual=r)).backward()
    got = [t.grad for t in (x, w, r)]
    plain = [t.detach().clone().requires_grad_() for t in (x, w, r)]
    h = plain[0] + plain[2]
    loss(h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * plain[1], h).backward()
    for a, b in zip(got, plain):
        if b.grad is None:
            assert torch.all(a == 0)
        else:
            assert torch.all((a - b.grad).abs() <= 1e-13 * (1 + b.grad.abs()))  # a few roundings of 1.1e-16 each
    assert len(norm_on_host) == use_y
    if use_y:
        assert (norm_on_host[0][1] is not None) == use_sum


def test_the_package_does_without_the_extension():
    """_fast.so missing, or built against another torch: a warning, and every call goes the general way."""
    code = """
import sys, warnings
sys.modules["late_interaction_retrieval_amd._fast"] = None  # an import of it raises ImportError
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from late_interaction_retrieval_amd import binding as bd
assert any("_fast.so" in str(w.message) for w in seen)
import torch
x, q = torch.zeros(4, 128), torch.zeros(4, 128).to(torch.float8_e4m3fn)
tab = bd.AdamWTensors.zeros([torch.zeros(5)])
for f in (lambda: bd.maxsim_rmsnorm_fwd(x), lambda: bd.maxsim_rmsnorm_bwd(x, x, x[:, 0]), lambda: bd.maxsim_quant_fp8(x),
          lambda: bd.maxsim_gemm_fp8(q, x[:, :1], q, x[:, :1]), lambda: bd.maxsim_adamw(tab, [torch.zeros(5)], 1)):
    try:
        f()
    except ValueError as e:
        assert "must be on the device" in str(e), e
    else:
        raise AssertionError("a host tensor was taken")
print("all general")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and "all general" in r.stdout, r.stderr


def test_a_linear_layer_refuses_what_its_backward_could_not_do():
    """More tokens, or columns, than the gradient's product takes along its sum: refused by the forward, where that
    gradient is asked for."""
    many = (1 << 22) + 1
    flat = lambda rows, grad: torch.zeros(rows, 16, requires_grad=grad)  # noqa: E731
    with pytest.raises(ValueError, match="no gradient of a weight"):
        bd.linear_fp8(flat(many, False), flat(3, True))
    with pytest.raises(ValueError, match="no gradient of x"):
        bd.linear_fp8(flat(3, True), flat(many, False))
    # not asked for, or within the limit: on to the call, which refuses host tensors
    for x, w in ((flat(many, True), flat(3, False)), (flat(3, False), flat(many, True)), (flat(many - 1, True), flat(3, True))):
        with pytest.raises(ValueError, match="must be on the device"):
            bd.linear_fp8(x, w)
    with torch.no_grad(), pytest.raises(ValueError, match="must be on the device"):
        bd.linear_fp8(flat(many, False), flat(3, True))


@pytest.mark.parametrize("shape", [(8,), (1, 8), (1, 1, 8), (2, 4)])
def test_a_gain_of_any_shape_gets_its_gradient(norm_on_host, shape):
    """The forward takes a gain of H contiguous values whatever their shape, and its gradient has that shape."""
    w = torch.ones(shape, dtype=torch.float64, requires_grad=True)
    x = torch.arange(24, dtype=torch.float64).reshape(3, 8)
    bd.rms_norm(x, w).sum().backward()
    xh = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    assert w.grad.shape == shape and torch.all((w.grad.reshape(-1) - xh.sum(0)).abs() <= 1e-13)


@pytest.mark.parametrize("state", [torch.float32, torch.float8_e4m3fn], ids=str)
@pytest.mark.parametrize("how", ["deepcopy", "file", "copy"])
def test_a_copied_optimiser_table_is_one_of_its_own(state, how):
    """Copied, or written and read back: the table names the copy's tensors, at an address that is its own."""
    tab = bd.AdamWTensors.zeros([torch.nn.Parameter(torch.ones(5).bfloat16()), torch.ones(300).bfloat16()], state)
    if how == "file":
        f = io.BytesIO()
        torch.save(tab, f)
        f.seek(0)
        other = torch.load(f, weights_only=False)  # written just now
    else:
        other = copy.deepcopy(tab) if how == "deepcopy" else copy.copy(tab)
    other._check_memory()
    assert other._address == other._table.ctypes.data != tab._address
    assert [int(a) for a in other._table["param"]] == [p.data_ptr() for p in other.params]
    assert [int(a) for a in other._table["m"]] == [p.data_ptr() for p in other.m]
    assert (other.params[1].data_ptr() == tab.params[1].data_ptr()) == (how == "copy")
    assert other.sizes == tab.sizes and (other.state_code, other.param_code) == (tab.state_code, tab.param_code)
    for a, b in zip(other._held, tab._held):
        assert a.dtype == b.dtype and torch.equal(a.float(), b.float())


def test_sizes_past_32_bits_are_refused():
    """2^32 + 5 rows would be 5 of them in the C call.  (Tensors without memory: the refusal comes before any use.)"""
    big = (1 << 32) + 5
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    e4m3 = torch.float8_e4m3fn
    x, wide = empty(big, 16), empty(2, big)
    q, few = empty(big, 16, dtype=e4m3), empty(4, 16, dtype=e4m3)
    one = empty(1, 1, dtype=torch.float32)
    raw = {n: getattr(bd, n).__wrapped__ for n in ("_rmsnorm_fwd", "_rmsnorm_bwd", "_quant_fp8", "_gemm_fp8")}
    for t in (x, wide):
        calls = [lambda: raw["_rmsnorm_fwd"](t, None, 1e-6, None, None, False, None, None, None, None),
                 lambda: raw["_rmsnorm_bwd"](t, t, t, None, None, False, None, None, None),
                 lambda: raw["_quant_fp8"](t, 1, True, False)]
        for call in calls:
            with pytest.raises(ValueError, match="32 bits"):
                call()
    for a, b in ((q, few), (few, q), (empty(4, big, dtype=e4m3), empty(4, big, dtype=e4m3))):
        with pytest.raises(ValueError, match="32 bits"):
            raw["_gemm_fp8"](a, one, b, one, torch.bfloat16, None, None)
    tab = bd.AdamWTensors.zeros([torch.zeros(5)])
    for step in (big, -big):
        with pytest.raises(ValueError, match="32 bits"):
            bd._adamw.__wrapped__(tab, [torch.zeros(5)], step, 1e-3, 0.9, 0.99, 1e-8, 0.0, None)
