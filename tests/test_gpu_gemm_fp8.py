"""The block-scaled FP8 product against the 64-bit form (tolerances:
encoder_ref.gemm_tolerance).  Run on an MI355X: pytest -m gpu."""
import numpy as np
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


def operand(seed, rows, K, extra=0):
    """[rows, K] e4m3 in rows a multiple of 16 bytes apart; NaN in every byte that does not count."""
    g = torch.Generator().manual_seed(seed)
    pitch = -(-K // 16) * 16 + extra
    buf = torch.full((rows, pitch), 0x7F, dtype=torch.uint8)
    buf[:, :K] = torch.randn(rows, K, generator=g).mul(100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return buf.to(DEV).view(torch.float8_e4m3fn)[:, :K]


def scales(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).uniform(0.2, 3.0, shape)).float().to(DEV)


def run(bd, M, N, K, b_rows, dtype, extra=0, **kw):
    a, b = operand(M + K, M, K, extra), operand(N + K + 1, N, K, extra)
    kb = -(-K // 128)
    sa, sb = scales(1, M, kb), scales(2, -(-N // b_rows), kb)
    c = bd.maxsim_gemm_fp8(a, sa, b, sb, out_dtype=dtype, **kw)
    return c, (a, sa, b, sb)


def check(c, a, sa, b, sb, b_rows, where=""):
    want, size, largest = ref.gemm(a, sa, b, sb, b_rows)
    got = c.double().cpu()
    tol = ref.gemm_tolerance(want, size, largest, a.shape[1], c.dtype)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d off, first %s, worst %.3g of its tolerance" % (
        where, int(bad.sum()), torch.nonzero(bad)[0].tolist(), float(((got - want).abs() / tol).max()))


# few rows (each count of 16), tiles with ends inside them, K with ends inside a block and a chunk, K split
SHAPES = [(1, 1, 1), (1, 128, 128), (2, 16, 16), (16, 17, 130), (17, 100, 1000), (33, 129, 384), (49, 200, 2049), (64, 15, 777),
          (65, 1, 128), (65, 129, 129), (128, 128, 2048), (100, 300, 4097), (200, 257, 31), (300, 130, 640),
          (130, 5, 20000), (256, 256, 255), (700, 384, 1024)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_product(bd, M, N, K, b_rows, dtype):
    if b_rows == 128 and N == 1:
        b_rows = 1  # the same scales
    c, ops = run(bd, M, N, K, b_rows, dtype)
    check(c, *ops, b_rows)
    again = bd.maxsim_gemm_fp8(*ops, out_dtype=dtype)
    assert torch.equal(again, c)


@pytest.mark.parametrize("M,N,K", [(3000, 2900, 300), (2817, 4096, 1040), (33000, 128, 200), (512, 20000, 100)])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_many_tiles(bd, M, N, K, b_rows):
    for dtype in (torch.float16, torch.float32):
        c, ops = run(bd, M, N, K, b_rows, dtype)
        if dtype == torch.float16:  # inputs to 448: keep the products inside fp16
            ops = (ops[0], ops[1] * 1e-3, ops[2], ops[3])
            c = bd.maxsim_gemm_fp8(*ops, out_dtype=dtype)
        rows = torch.from_numpy(np.unique(np.random.default_rng(3).integers(0, M, 40)))
        rows = torch.cat([rows, torch.tensor([M - 1])])
        check(c[rows.to(DEV)], ops[0].view(torch.uint8)[rows.to(DEV)].view(torch.float8_e4m3fn), ops[1][rows.to(DEV)],
              ops[2], ops[3], b_rows)


@pytest.mark.parametrize("M", [5, 150])
def test_pitches(bd, M):
    """Wider pitches than K, and an output inside a larger one: nothing else is written."""
    N, K = 37, 200
    _, ops = run(bd, M, N, K, 128, torch.float16, extra=48)
    ops = (ops[0], ops[1] * 1e-3, ops[2], ops[3])
    for dtype in (torch.float16, torch.float32):
        big = torch.full((M + 2, N + 6), 7, dtype=dtype, device=DEV)
        into = big[1:-1, 3:3 + N]
        bd.maxsim_gemm_fp8(*ops, out=into)
        check(into, *ops, 128)
        big[1:-1, 3:3 + N] = 7
        assert torch.all(big == 7)


def test_exact_small_integers(bd):
    """Small whole numbers and scales that are powers of two: every product and sum is exact, in every kernel, so
    that a wrong row, column, block or scale shows whatever the tolerance."""
    g = torch.Generator().manual_seed(1)
    for M, N, K in ((7, 40, 300), (60, 130, 513), (200, 140, 1100), (2300, 2100, 260)):
        a = torch.randint(-2, 3, (M, K), generator=g).float()
        b = torch.randint(-2, 3, (N, K), generator=g).float()
        kb = -(-K // 128)
        for b_rows in (1, 128):
            sa = torch.exp2(torch.randint(-1, 2, (M, kb), generator=g).float())
            sb = torch.exp2(torch.randint(-1, 2, (-(-N // b_rows), kb), generator=g).float())
            pad = -K % 16
            qa = torch.nn.functional.pad(a, (0, pad)).to(torch.float8_e4m3fn).to(DEV)[:, :K]
            qb = torch.nn.functional.pad(b, (0, pad)).to(torch.float8_e4m3fn).to(DEV)[:, :K]
            want = (a * sa.repeat_interleave(128, 1)[:, :K]).double() @ (
                b * ref.spread(sb, b_rows, 128, (N, K))).double().t()
            c = bd.maxsim_gemm_fp8(qa, sa.to(DEV), qb, sb.to(DEV), out_dtype=torch.float32)
            assert torch.equal(c.double().cpu(), want), (M, N, K, b_rows)
            c = bd.maxsim_gemm_fp8(qa, sa.to(DEV), qb, sb.to(DEV), out_dtype=torch.bfloat16)
            assert torch.equal(c.cpu(), want.to(torch.bfloat16)), (M, N, K, b_rows)


def test_empty_and_nan(bd):
    one = lambda *s: torch.ones(s, device=DEV)  # noqa: E731
    for M in (3, 100):
        a, b = operand(1, M, 0), operand(2, 9, 0)
        c = bd.maxsim_gemm_fp8(a, one(M, 0), b, one(1, 0))
        assert c.shape == (M, 9) and torch.all(c == 0)
        assert bd.maxsim_gemm_fp8(operand(1, 0, 32), one(0, 1), operand(1, 4, 32), one(4, 1)).shape == (0, 4)
        a, b = operand(1, M, 160), operand(2, 140, 160)
        sa = one(M, 2)
        sa[1, 1] = float("nan")       # a block that was not finite: its row, and no other
        for dtype in (torch.bfloat16, torch.float32):
            c = bd.maxsim_gemm_fp8(a, sa, b, one(2, 2), out_dtype=dtype)
            assert torch.isnan(c[1]).all() and torch.isfinite(c[0]).all() and torch.isfinite(c[2:]).all()


def test_refusals(bd):
    a, b, s = operand(1, 4, 128), operand(2, 6, 128), torch.ones(4, 1, device=DEV)
    one = torch.ones(1, 1, device=DEV)
    with pytest.raises(ValueError):
        bd.maxsim_gemm_fp8(a, s, operand(2, 6, 64), one)
    with pytest.raises(ValueError):
        bd.maxsim_gemm_fp8(a, s[:3], b, one)
    with pytest.raises(ValueError):
        bd.maxsim_gemm_fp8(a, s, b, torch.ones(2, 1, device=DEV))
    with pytest.raises(TypeError):
        bd.maxsim_gemm_fp8(a.view(torch.int8), s, b, one)
    with pytest.raises(TypeError):
        bd.maxsim_gemm_fp8(a, s, b, one, out_dtype=torch.int32)
    with pytest.raises(bd.MaxSimError):      # rows 100 bytes apart
        bd.maxsim_gemm_fp8(torch.zeros(600, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:400].reshape(4, 100),
                           s, operand(1, 6, 100), one)
    tight = torch.zeros(3 * 112 + 100, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).as_strided((4, 100), (112, 1))
    with pytest.raises(ValueError):          # the last row ends before K rounded up to 16
        bd.maxsim_gemm_fp8(tight, s, operand(1, 6, 100), one)
    big = [operand(1, 128, 1 << 16), torch.ones(128, 512, device=DEV)]
    with pytest.raises(bd.MaxSimError):
        bd.maxsim_gemm_fp8(*big, *big, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("N", [1 << 26, (1 << 27) + 5])
def test_one_row_by_very_many(bd, N):
    """More rows of B than one launch of the kernel for few rows of A holds threads for."""
    codes = torch.arange(33, 94, dtype=torch.uint8, device=DEV)  # positive normal values
    B = codes.repeat(N * 16 // 61 + 1)[:N * 16].view(torch.float8_e4m3fn).view(N, 16)
    A = torch.full((1, 16), 0.5, device=DEV).to(torch.float8_e4m3fn)
    one = torch.ones(1, 1, device=DEV)
    sb = torch.arange(1, -(-N // 128) + 1, device=DEV).remainder_(7).add_(1).float().unsqueeze(1)
    c = bd.maxsim_gemm_fp8(A, one, B, sb, out_dtype=torch.bfloat16)
    for at in (0, 12345 * 128, (1 << 26) - 300, N - 200):
        want = B[at:at + 200].double().sum(1) * 0.5
        want = want * sb[:, 0].double()[torch.arange(at, min(at + 200, N), device=DEV) // 128]
        got = c[0, at:at + 200].double()
        # one rounding to bf16, and 16 products that the matrix cores add to 13 bits below the largest
        assert torch.all((got - want).abs() <= want.abs() * (2.0 ** -8 * 1.01 + 16 * 2.0 ** -13)), at
