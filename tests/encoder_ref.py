"""Plain 64-bit forms of the embedding head's operators (torch on the CPU, not
collected by pytest), and the error bounds that the tests hold the kernels to.

Bounds.  u = 2^-24 is the rounding of one fp32 operation.  A sum of n terms
added in any order is off by at most n u times the sum of magnitudes.  A value
stored in a type is off by at most eps(type) / 2 relative to itself.
"""
import torch

U = 2.0 ** -24
TOP = {"e4m3": 448.0, "i8": 127.0}
TINY = 2.0 ** -100


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def round_e4m3(t):
    """Nearest e4m3 value (ties to even), |t| <= 464."""
    _, e = torch.frexp(t)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(t / step) * step


def blocks(y, br, bc):
    """y [R, C] cut into [R/br, br, C/bc, bc], zeros where it does not fill them."""
    R, C = y.shape
    full = y.new_zeros(-(-R // br) * br, -(-C // bc) * bc)
    full[:R, :C] = y
    return full.reshape(full.shape[0] // br, br, full.shape[1] // bc, bc)


def spread(scale, br, bc, shape):
    """A scale for each value from a scale for each block."""
    return scale.repeat_interleave(br, 0).repeat_interleave(bc, 1)[:shape[0], :shape[1]]


def check_held(q, scale, y, br, bc, kind, err=0.0, where=""):
    """Codes q and scales hold y [R, C] (64 bits) in blocks of br x bc: the scale is the block's, and each value is a
    nearest one.  err: how far the values that were rounded may be from y, relative to each and to the block's largest
    (0 for values that the kernel reads exactly)."""
    q, scale, y = q.double().cpu(), scale.double().cpu(), y.cpu()
    top = blocks(y, br, bc).abs().amax(dim=(1, 3))
    zero = top < TINY * (1 + 1e-6)
    want = torch.where(zero, torch.ones_like(top), top / TOP[kind])
    scale = scale.reshape(want.shape)
    assert torch.all((scale - want).abs() <= want * (err + 2 * U)), where + ": scale"
    s = spread(scale, br, bc, y.shape)
    t = y / s
    assert torch.all(q[spread(zero.double(), br, bc, y.shape) > 0] == 0), where + ": blocks held as zeros"
    if kind == "i8":
        step = torch.ones_like(t)
    else:
        _, e = torch.frexp(t.abs().clamp_max(TOP[kind]))
        step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    # half a step, the division's rounding, and what y itself may be off
    tol = step / 2 + t.abs() * (4 * U + err) + TOP[kind] * err
    bad = (q - t).abs() > tol
    assert not bad.any(), "%s: %d values are not the nearest, first at %s" % (where, int(bad.sum()),
                                                                           torch.nonzero(bad)[0].tolist())


def rmsnorm(x, weight, residual, eps):
    h = x.double() + (0 if residual is None else residual.double())
    r = 1 / torch.sqrt((h * h).mean(-1) + eps)
    y = h * r[..., None] * (1 if weight is None else weight.double())
    return h, r, y


def rmsnorm_bwd(dy, h, r, weight, dsum):
    """dx, dweight, and for each the sum of magnitudes that its rounding errors are relative to."""
    dy, h, r = dy.double(), h.double(), r.double()[:, None]
    g = dy * (1 if weight is None else weight.double())
    xh = h * r
    mean = (g * xh).mean(1, keepdim=True)
    size = (g * xh).abs().mean(1, keepdim=True)
    dx = r * (g - xh * mean) + (0 if dsum is None else dsum.double())
    dx_size = r * (g.abs() + xh.abs() * size) + (0 if dsum is None else dsum.double().abs())
    return dx, (dy * xh).sum(0), dx_size, (dy * xh).abs().sum(0)


def gemm(a, a_scale, b, b_scale, b_rows):
    """c, the sum of magnitudes, and the sum over blocks of the largest scaled product."""
    M, K = a.shape
    N = b.shape[0]
    c = torch.zeros(M, N, dtype=torch.float64)
    size, largest = torch.zeros_like(c), torch.zeros_like(c)
    a, b, a_scale, b_scale = a.float().double().cpu(), b.float().double().cpu(), a_scale.double().cpu(), b_scale.double().cpu()
    rows = torch.arange(N) // b_rows
    for kb in range(-(-K // 128)):
        x, w = a[:, kb * 128:(kb + 1) * 128], b[:, kb * 128:(kb + 1) * 128]
        s = a_scale[:, kb, None] * b_scale[rows, kb][None]
        c += s * (x @ w.t())
        size += s.abs() * (x.abs() @ w.abs().t())
        largest += s.abs() * x.abs().amax(1)[:, None] * w.abs().amax(1)[None]
    return c, size, largest


def gemm_tolerance(c, size, largest, K, dtype):
    """One rounding to the result's type, fp32 sums, and for 16-bit results the 8-bit instruction, which keeps at least
    12 bits below a block's largest product."""
    tol = half_step(dtype) * c.abs() + (128 + K / 128 + 4) * U * size
    if dtype != torch.float32:
        tol = tol + 2.0 ** -12 * largest
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half of the smallest step
    return tol


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd):
    p, g = p.double(), g.double()
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    return p - lr * wd * p - lr * step, m, v
