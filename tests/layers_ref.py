"""Plain 64-bit forms of the attention layer's operators and of the distillation loss (torch on the CPU, not collected by
pytest), and the error bounds that the tests hold the kernels to.

Bounds.  u = 2^-24 is the rounding of one fp32 operation; a sum of n terms in any order is off by at most n u times the
sum of magnitudes; rounding to a type is off by half a step, finfo.eps / 2 of the value (for fp16 also 2^-25, half of its
smallest step).  Errors are carried through the formulas to first order, by magnitudes.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of fp16's smallest step; of the wider types the smallest normal value of fp32, 2^-126, below which an exponential
    or a product may be held as 0."""
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126


# ---------------------------------------------------------------- rotary positions


def rope(x, inv_freq, positions, layout, scale, inverse=False):
    """(y, bound) of x [T, H, D] at positions [T], both 64 bits."""
    dtype, x, half = x.dtype, x.double(), inv_freq.numel()
    a = positions.double()[:, None] * inv_freq
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    if inverse:
        s = -s
    y, size = x.clone(), torch.zeros_like(x)
    left, right = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    u, w = x[..., left], x[..., right]
    y[..., left], y[..., right] = scale * (u * c - w * s), scale * (w * c + u * s)
    size[..., left] = size[..., right] = abs(scale) * (u.abs() + w.abs())
    # the angle: fp64 to 1e-15 of the turns, then 2^-25 of half a turn (pi); the sine and cosine themselves 4 units; the
    # factor's product, and two products and a sum
    angle = 4 * a.abs().max().item() * 2.0 ** -52 + math.pi * 2.0 ** -24
    return y, size * (angle + 9 * U) + half_step(dtype) * y.abs() + tiny(dtype)


# ---------------------------------------------------------------- attention


def seen(nq, nk, window, sinks):
    """[nq, nk]: which keys a query sees."""
    p, j = torch.arange(nq)[:, None] + nk - nq, torch.arange(nk)[None]
    vis = torch.ones(nq, nk, dtype=torch.bool)
    if window[1] >= 0:
        vis &= j <= p + window[1]
    if window[0] >= 0:
        vis &= (j >= p - window[0]) | (j < sinks)
    return vis


def one_head(q, k, v, vis, scale, g=None, exact_rest=True):
    """{name: (value, bound)} of one head's rows: out, lse and, with the gradient g of out, dq, dk, dv (before a shared
    head's are added up)."""
    T = q.dtype
    h, tn = half_step(T), tiny(T)
    q, k, v = q.double(), k.double(), v.double()
    n, D = k.shape
    s, a = scale * q @ k.t(), scale * q.abs() @ k.abs().t()
    s = s.masked_fill(~vis, -math.inf)
    size = s.abs().masked_fill(~vis, 0.0)
    blind = ~vis.any(1)
    top = s.amax(1) if n else torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    e = torch.exp(s - torch.where(blind, 0.0, top)[:, None])
    total = e.sum(1)
    p = e / torch.where(blind, 1.0, total)[:, None]
    lse = torch.where(blind, -math.inf, top + torch.log(total))
    most = size.amax(1) if n else torch.zeros(q.shape[0], dtype=torch.float64)
    # a score: D products; the scale's rounding, the reference's product and the sum of the exponent; the exponential
    es = ((D + 4) * U * a).masked_fill(~vis, 0.0) + 6 * U * most[:, None] + 8 * U
    e_row = es.amax(1) if n else torch.zeros(q.shape[0], dtype=torch.float64)
    pv = p @ v.abs()
    o = p @ v
    # P rounded to T (fp16: to a step of 2^-24 at least, where the largest is 1 or more); sums of n terms, 64 joined parts
    off = (h + 2 * e_row[:, None] + (2 * n + 80) * U) * pv + tn * vis.double() @ v.abs()
    out = {"out": (o, off + h * o.abs() + tn),
           "lse": (lse, e_row + (n + 80) * U + 4 * U * torch.where(blind, 0.0, lse.abs()) + 4 * U)}
    if g is None:
        return out
    g = g.double()
    dp, adp = g @ v.t(), g.abs() @ v.abs().t()
    delta = (g * o).sum(1, keepdim=True)
    off_o = off + (h * h * o.abs() + tn if exact_rest else h * o.abs() + tn)
    e_delta = (g.abs() * off_o).sum(1, keepdim=True) + (D + 4) * U * (g.abs() * o.abs()).sum(1, keepdim=True)
    ds = p * (dp - delta)
    ep = es + 4 * U * (size + torch.where(blind, 0.0, lse.abs())[:, None]) + torch.where(blind, 0.0, out["lse"][1])[:, None]
    e_ds = p * (ep * (dp - delta).abs() + (D + 4) * U * adp + e_delta + 3 * U * (dp.abs() + delta.abs())) + h * ds.abs()
    low = vis.double() * tn  # fp16: half a step of its smallest values, in the scale of the row's (or largest) dO
    row_top = g.abs().amax(1, keepdim=True)
    if T != torch.float16:
        row_top = row_top.clamp_min(1.0)
    dq = scale * ds @ k
    out["dq"] = (dq, scale * (e_ds + low * row_top + (n + 4) * U * ds.abs()) @ k.abs() + (h + 4 * U) * dq.abs() + tn)
    dk = scale * ds.t() @ q
    m = q.shape[0]
    out["dk"] = (dk, scale * (e_ds + low * row_top.max() + (m + 4) * U * ds.abs()).t() @ q.abs() + 4 * U * dk.abs())
    dv = p.t() @ g
    out["dv"] = (dv, (p * (h + ep + (m + 4) * U) + low / 256).t() @ g.abs() + 4 * U * dv.abs())
    return out


def attention(q, k, v, lens, scale, window, sinks, g=None, rows=None, exact_rest=True):
    """{name: (value, bound)} for CPU tensors [rows, H, D] with lens a list of (first q row, queries, first k row, keys);
    rows of no sequence are zeros with bound 0."""
    Hq, Hk = q.shape[1], k.shape[1]
    G = Hq // Hk
    names = ["out", "lse"] + (["dq", "dk", "dv"] if g is not None else [])
    shape = {"out": q.shape, "lse": q.shape[:2], "dq": q.shape, "dk": k.shape, "dv": k.shape}
    got = {n: (torch.zeros(shape[n], dtype=torch.float64), torch.zeros(shape[n], dtype=torch.float64)) for n in names}
    for q0, nq, k0, nk in lens:
        vis, qs, ks = seen(nq, nk, window, sinks), slice(q0, q0 + nq), slice(k0, k0 + nk)
        if nq == 0:
            continue
        for hd in range(Hq):
            r = one_head(q[qs, hd], k[ks, hd // G], v[ks, hd // G], vis, scale, None if g is None else g[qs, hd], exact_rest)
            for n in names:
                for i in (0, 1):
                    if n in ("dk", "dv"):
                        got[n][i][ks, hd // G] += r[n][i]
                    else:
                        got[n][i][qs, hd] = r[n][i]
    if g is not None:  # the shared heads' sum, rounded once
        for n in ("dk", "dv"):
            value, bound = got[n]
            bound += (half_step(q.dtype) + G * U) * value.abs() + tiny(q.dtype) * (bound > 0)
    return got


def check(got, want, where):
    value, bound = want
    got = got.double().cpu().reshape(value.shape)
    same = torch.where(torch.isfinite(value), torch.isfinite(got), got == value)
    assert same.all(), "%s: %d values not finite, or not where they should be" % (where, int((~same).sum()))
    d = torch.where(torch.isfinite(value), (got - value).abs(), 0.0)
    bad = d > torch.where(torch.isfinite(value), bound, 0.0)
    assert not bad.any(), "%s: %d of %d values out of bounds, first at %s: %g for %g, bound %g" % (
        where, int(bad.sum()), bad.numel(), torch.nonzero(bad)[0].tolist(), got[bad][0], value[bad][0], bound[bad][0])


# ---------------------------------------------------------------- distillation


def distill(z, index, teacher, T, dloss=None):
    """{loss, dscores: (value, bound)} of z [N, V] with entries index, teacher [N, K]."""
    dtype, z, t = z.dtype, z.double(), teacher.double()
    N, V = z.shape
    K = index.shape[1]
    ok = (index >= 0) & (index < V)
    lp = torch.log_softmax(z / T, 1) if V else z
    lp = lp.masked_fill(z == -math.inf, -math.inf)
    at = index.long().clamp(0, max(V - 1, 0))
    masked = (t / T).masked_fill(~ok, -math.inf)
    none = ~torch.isfinite(masked).any(1) if K else torch.ones(N, dtype=torch.bool)
    lq = torch.log_softmax(masked.masked_fill(none[:, None], 0.0), 1)
    q = torch.where(none[:, None] | ~ok, 0.0, lq.exp())
    terms = torch.where(q > 0, lq - (lp.gather(1, at) if V else 0.0), 0.0)
    loss = T * T * (q * terms).sum(1)
    spread = z.masked_fill(z == -math.inf, math.nan)
    wide = torch.nan_to_num((z.amax(1, keepdim=True) - spread) / T, 0.0).clamp_min(0) if V else z  # exponents
    t_wide = torch.where(ok & torch.isfinite(t), masked.amax(1, keepdim=True) - masked, 0.0) if K else t
    out = {"loss": (loss, None)}
    # exponents: a difference, the factor and a product; sums of V and K; logarithms; the terms' sum
    e_q = 8 * U * (1 + t_wide) + (K + 4) * U + 8 * U
    e_p = 8 * U * (1 + torch.where(ok, wide.gather(1, at), 0.0) if V else t_wide) + (V + 4) * U + 8 * U * math.log(max(V, 2))
    fin = torch.where(torch.isfinite(terms), terms.abs(), 0.0)
    out["loss"] = (loss, T * T * (q * (fin * e_q + e_q + e_p + 8 * U * (lq.abs().nan_to_num(0, 0, 0)
                   + torch.where(torch.isfinite(terms), (terms - lq).abs(), 0.0).nan_to_num(0, 0, 0)))
                   + (K + 4) * U * q * fin).sum(1) + 1e-37)
    if dloss is not None:
        p = lp.exp() if V else z
        if V:
            p = torch.where((z == -math.inf).all(1, keepdim=True), 0.0, p)
        w = torch.where(none, 0.0, dloss.double() * T)[:, None]
        qs, eq = torch.zeros_like(z), torch.zeros_like(z)
        for n in range(N):
            for k in range(K):
                if ok[n, k]:
                    qs[n, at[n, k]] += q[n, k]
                    eq[n, at[n, k]] += q[n, k] * e_q[n, k]
        d = w * (p - qs)
        e = w.abs() * (p * (8 * U * (1 + wide) + (V + 4) * U + 8 * U * math.log(max(V, 2))) + eq + (K + 4) * U * (p + qs))
        out["dscores"] = (d, e + (half_step(dtype) + 2 * U) * d.abs() + tiny(dtype))
    return out
