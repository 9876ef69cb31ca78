"""Rows in e4m3 with a scale for each 128 values, as rows, transposed and in
128 x 128 blocks, against the 64-bit form.  The kernel reads the values exactly,
so every code is a nearest one up to the rounding of scale and division.
Run on an MI355X: pytest -m gpu."""
import numpy as np
import pytest
import torch

import encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def bd():
    from late_interaction_retrieval_amd import binding
    assert torch.cuda.is_available()
    return binding


def values(seed, R, C, dtype):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.standard_normal((R, C)) * np.exp2(g.integers(-6, 6, (R, 1)))).to(dtype)


SHAPES = [(1, 1), (1, 128), (128, 1), (3, 7), (128, 128), (129, 127), (127, 129), (16, 256), (300, 200), (1, 1000),
          (1000, 1), (257, 385)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_blocks(bd, R, C, dtype):
    x = values(R * 7 + C, R, C, dtype)
    for br in (1, 128):
        q, s, qt, st = bd.maxsim_quant_fp8(x.to(DEV), block_rows=br, transposed=True)
        assert q.shape == (R, C) and qt.shape == (C, R) and q.stride(0) % 16 == 0 and qt.stride(0) % 16 == 0
        ref.check_held(q, s, x.double(), br, 128, "e4m3", 0.0, "rows")
        ref.check_held(qt, st, x.double().t(), br, 128, "e4m3", 0.0, "transposed")
        if br == 128:
            assert torch.equal(q.float(), qt.float().t()) and torch.equal(s, st.t())
        only = bd.maxsim_quant_fp8(x.to(DEV), block_rows=br)
        assert torch.equal(only[0].float(), q.float()) and torch.equal(only[1], s) and only[2] is None
        only = bd.maxsim_quant_fp8(x.to(DEV), block_rows=br, rows=False, transposed=True)
        assert torch.equal(only[2].float(), qt.float()) and torch.equal(only[3], st) and only[0] is None


def test_slices_and_ends(bd):
    """A slice of wider rows at an odd element; the bytes between the width and the pitch are left alone."""
    wide = values(3, 70, 300, torch.float16).to(DEV)
    x = wide[::2, 37:37 + 150]
    q, s, qt, st = bd.maxsim_quant_fp8(x, transposed=True)
    ref.check_held(q, s, x.double().cpu(), 1, 128, "e4m3", 0.0, "slice")
    ref.check_held(qt, st, x.double().cpu().t(), 1, 128, "e4m3", 0.0, "slice transposed")
    lib, R, C = bd.lib(), x.shape[0], x.shape[1]
    buf = torch.full((R + 2, 160), 0x55, dtype=torch.uint8, device=DEV)
    bt = torch.full((C + 2, 48), 0x55, dtype=torch.uint8, device=DEV)
    sc, sct = torch.empty_like(s), torch.empty_like(st)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.maxsim_quant_fp8(x.data_ptr(), 600, R, C, 0, 1, buf[1:].data_ptr(), 160, sc.data_ptr(), bt[1:].data_ptr(),
                                48, sct.data_ptr(), stream) == 0
    assert torch.equal(buf[1:-1, :C], q.view(torch.uint8)) and torch.equal(bt[1:-1, :R], qt.view(torch.uint8))
    buf[1:-1, :C] = 0x55
    bt[1:-1, :R] = 0x55
    assert torch.all(buf == 0x55) and torch.all(bt == 0x55)


def test_extremes(bd):
    x = torch.zeros(4, 256)
    x[0, :128] = 2.0 ** -101          # below the smallest block: zeros, scale 1
    x[0, 128:] = 2.0 ** -100
    x[1, 3] = float("nan")
    x[1, 200] = -float("inf")
    x[2] = 3e38
    x[3, 0], x[3, 1] = 448.0, 448.0 * 2 ** -20  # one value far below its block's largest
    q, s, _, _ = bd.maxsim_quant_fp8(x.to(DEV))
    q, s = q.float().cpu(), s.cpu()
    assert s[0, 0] == 1 and torch.all(q[0, :128] == 0) and torch.all(q[0, 128:] == 448)
    assert torch.isnan(s[1]).all() and torch.all(q[1] == 0)
    assert torch.all(q[2] == 448) and abs(float(s[2, 0]) / (3e38 / 448) - 1) < 1e-6
    assert q[3, 0] == 448 and q[3, 1] == 0 and s[3, 0] == 1 and s[3, 1] == 1
    for shape in ((0, 5), (5, 0)):
        q, s, qt, st = bd.maxsim_quant_fp8(torch.zeros(shape, device=DEV), transposed=True)
        assert q.shape == shape and qt.shape == shape[::-1]


def test_every_code(bd):
    """Values on and halfway between the codes (scale 1): nearest, ties to even, as torch rounds them."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[torch.isfinite(codes)].sort().values.unique()
    x = torch.cat([codes, (codes[1:] + codes[:-1]) / 2, torch.tensor([448.0])])
    x = torch.nn.functional.pad(x, (0, -x.numel() % 127)).reshape(-1, 127)
    x = torch.nn.functional.pad(x, (0, 1), value=448.0)  # every block's largest: scale 1
    q, s, _, _ = bd.maxsim_quant_fp8(x.to(DEV))
    assert torch.all(s == 1)
    assert torch.equal(q.float().cpu(), x.to(torch.float8_e4m3fn).float())


def test_refusals(bd):
    x = torch.zeros(4, 128, device=DEV)
    with pytest.raises(ValueError):
        bd.maxsim_quant_fp8(x[0])
    with pytest.raises(ValueError):
        bd.maxsim_quant_fp8(x, rows=False)
    with pytest.raises(ValueError):
        bd.maxsim_quant_fp8(x.t())
    with pytest.raises(TypeError):
        bd.maxsim_quant_fp8(x.double())
    with pytest.raises(bd.MaxSimError):
        bd.maxsim_quant_fp8(x, block_rows=64)
