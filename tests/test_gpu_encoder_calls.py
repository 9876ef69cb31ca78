"""How calls of the embedding head's operators are made and refused, with tensors on the device.
Run on an MI355X: pytest -m gpu."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


@pytest.fixture
def hip(bd):
    """The HIP runtime that this process has loaded."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64.so" in line}
    assert len(paths) == 1, paths
    return ctypes.CDLL(paths.pop())


@pytest.mark.parametrize("general", [False, True])
def test_an_old_error_does_not_repeat_a_step(bd, hip, general):
    """An error that an earlier call left unread is not the step's: one step is made, both ways of making the call."""
    where = dict(stream=torch.cuda.current_stream()) if general else {}
    p, g = torch.ones(300, device=DEV), torch.full((300,), 0.5, device=DEV)
    tab = bd.AdamWTensors.zeros([p])
    torch.cuda.synchronize()
    assert hip.hipSetDevice(4096) != 0
    bd.maxsim_adamw(tab, [g], 1, lr=0.125, beta1=0.5, beta2=0.5, weight_decay=0.0, **where)
    left = hip.hipGetLastError()
    torch.cuda.synchronize()
    assert left == 0
    # m = g / 2, v = g^2 / 2 after one step; each 3/4 of g and g^2 after a second
    assert torch.all(tab.m[0] == 0.25) and torch.all(tab.v[0] == 0.125)


def test_the_extension_names_its_status(bd):
    """Called with everything it takes: refusals of the library come back as its status, what the extension does not
    handle as None, and nothing moves."""
    tab = bd.AdamWTensors.zeros([torch.ones(70, device=DEV), torch.ones(300, device=DEV)], torch.float8_e4m3fn)
    g = [torch.ones(70, device=DEV), torch.ones(300, device=DEV)]

    def call(grads=g, beta1=0.9, step=1):
        return bd._fast.adamw(tab._address, 2, 0, tab.param_code, tab.state_code, tab._held, grads, 1e-3, beta1, 0.99, 1e-8,
                              0.0, step)

    assert call(g[:1]) is None and call([g[0], g[0]]) is None and call([g[0], g[1].bfloat16()]) is None
    assert call([t.cpu() for t in g]) is None and call(tuple(g)) is None and call(step=0) is None
    assert call(beta1=1.0) == 2                       # a size or a rate out of range
    assert all(torch.all(p == 1) for p in tab.params) and all(torch.all(m.float() == 0) for m in tab.m)
    versions = [p._version for p in tab.params]
    assert call() == 0
    assert all(torch.all(p < 1) for p in tab.params) and [p._version for p in tab.params] == [v + 1 for v in versions]
