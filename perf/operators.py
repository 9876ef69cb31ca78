"""The operators around MaxSim's operands, case by case: the embedding head that makes the token rows (RMS norm with
the residual's addition and an 8-bit output, quantisation, the block-scaled FP8 product) and the step that trains it
(the norm's backward, the FP8 gradient products, AdamW over many tensors).

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda:0"
BLOCK = 128  # columns (or rows) that share a scale
E4M3_MAX = 448.0
TINY = 2.0 ** -100  # a block whose largest magnitude is below this is held as zeros with scale 1
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8,
          "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 11


def listed():
    return [
        # one query's 32 token rows on their way into the int8 scan: the smallest call, latency alone
        {"name": "norm_query_i8", "op": "norm", "rows": 32, "width": 128, "dtype": "f32", "out": "i8",
         "residual": False, "rstd": False},
        # a batch of documents (32 of 1024 tokens) after the encoder's last layer: sum, norm, FP8 operand
        {"name": "norm_tokens_e4m3", "op": "norm", "rows": 32768, "width": 2048, "dtype": "bf16", "out": "e4m3",
         "residual": True, "rstd": True},
        # an odd batch of an odd width (a concatenation of features), fp16
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 1003, "width": 769, "dtype": "f16", "dsum": False},
        # the training step's tokens, with the gradient that arrives on the residual stream
        {"name": "norm_bwd_tokens", "op": "norm_bwd", "rows": 16384, "width": 2048, "dtype": "bf16", "dsum": True},
        # a projection's weight, 128 x 128 blocks, both layouts (once a step in training)
        {"name": "quant_weight", "op": "quant", "rows": 128, "cols": 2048, "dtype": "bf16", "block_rows": 128,
         "both": True},
        # a training step's activations, along the width for the forward and along the tokens for dW
        {"name": "quant_tokens", "op": "quant", "rows": 16384, "cols": 4096, "dtype": "bf16", "block_rows": 1,
         "both": True},
        # one query (32 tokens) through a hidden layer while a user waits: the weights' bytes
        {"name": "gemm_query", "op": "gemm", "m": 32, "n": 2048, "k": 2048, "b_rows": 128, "out": "bf16"},
        # documents projected to the embedding width while a corpus is indexed
        {"name": "gemm_project", "op": "gemm", "m": 65536, "n": 128, "k": 2048, "b_rows": 128, "out": "bf16"},
        # a hidden layer over a large batch of documents
        {"name": "gemm_hidden", "op": "gemm", "m": 16384, "n": 8192, "k": 4096, "b_rows": 128, "out": "bf16"},
        # a weight's gradient: both operands scaled along an odd number of tokens, fp32 out
        {"name": "gemm_dw", "op": "gemm", "m": 1024, "n": 2048, "k": 20001, "b_rows": 1, "out": "f32"},
        # the head alone: a 128-wide projection and two gains, fp32: latency
        {"name": "adamw_head", "op": "adamw", "tensors": 3, "total": 132224, "dtype": "f32", "state": "f32",
         "shape_seed": 1},
        # a small encoder's tensors of odd sizes: bf16 weights with fp32 masters, states in 8 bits
        {"name": "adamw_encoder_8bit", "op": "adamw", "tensors": 100, "total": 67108864, "dtype": "bf16",
         "state": "e4m3", "shape_seed": 2},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "quant", "gemm", "gemm", "gemm", "adamw"])
    if op == "norm":
        width = rng.choice([128, _spread(rng, 64, 8192), 8 * _spread(rng, 16, 1024)])
        return {"op": op, "rows": _spread(rng, 1, min(65536, (1 << 26) // width)), "width": width,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "out": rng.choice(["i8", "e4m3", "same"]),
                "residual": rng.random() < 0.6, "rstd": rng.random() < 0.5}
    if op == "norm_bwd":
        width = rng.choice([128, _spread(rng, 64, 8192), 8 * _spread(rng, 16, 1024)])
        return {"op": op, "rows": _spread(rng, 1, min(65536, (1 << 25) // width)), "width": width,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "dsum": rng.random() < 0.5}
    if op == "quant":
        cols = rng.choice([128, _spread(rng, 64, 8192), 16 * _spread(rng, 8, 512)])
        return {"op": op, "rows": _spread(rng, 1, min(32768, (1 << 26) // cols)), "cols": cols,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "block_rows": rng.choice([1, 1, 128]),
                "both": rng.random() < 0.6}
    if op == "gemm":
        n = rng.choice([128, 16 * _spread(rng, 8, 512), _spread(rng, 64, 8192)])
        k = rng.choice([16 * _spread(rng, 8, 1024), _spread(rng, 128, 16384)])
        return {"op": op, "m": _spread(rng, 1, min(65536, (1 << 38) // (n * k))), "n": n, "k": k,
                "b_rows": rng.choice([128, 128, 1]), "out": rng.choice(["bf16", "bf16", "f16", "f32"])}
    state = rng.choice(["f32", "e4m3"])
    return {"op": op, "tensors": _spread(rng, 1, 200), "total": _spread(rng, 4096, 1 << 26),
            "dtype": rng.choice(["f32", "bf16", "f16"]), "state": state, "shape_seed": rng.randrange(1 << 30)}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _hidden(g, rows, width, dtype, scale=1.0):
    """Rows as an encoder's layer gives them: normal, with a few channels of a larger spread."""
    x = torch.randn(rows, width, device=DEV, generator=g)
    spread = torch.where(torch.rand(width, device=DEV, generator=g) < 0.01, 8.0, 1.0)
    return (x * spread * scale).to(dtype)


def _e4m3(g, rows, k):
    """An FP8 operand and its scales, a scale for each 128 along k, in rows of a multiple of 16 bytes."""
    pitch = -(-k // 16) * 16
    x = torch.randn(rows, pitch, device=DEV, generator=g).mul_(110.0).clamp_(-E4M3_MAX, E4M3_MAX)
    return x.to(torch.float8_e4m3fn)[:, :k]


def _sizes(case):
    """The tensors' sizes: they add up to the total, odd ones among them."""
    n, total = case["tensors"], case["total"]
    r = torch.Generator()
    r.manual_seed(case["shape_seed"])
    share = torch.rand(n, generator=r, dtype=torch.float64) ** 3 + 1e-3
    sizes = [max(1, int(total * s)) for s in (share / share.sum()).tolist()]
    sizes[-1] = max(1, total - sum(sizes[:-1]))
    return sizes


def _flat_size(sizes):
    """Elements of the flat buffer that holds the tensors, each from a multiple of 128 on."""
    return sum(-(-n // BLOCK) * BLOCK for n in sizes)


def _views(flat, sizes, per=1):
    """The tensors in a flat buffer with a value for each `per` elements."""
    at, got = 0, []
    for n in sizes:
        got.append(flat[at // per:at // per + -(-n // per)])
        at += -(-n // BLOCK) * BLOCK
    return got


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        s = {"x": _hidden(g, case["rows"], case["width"], dt),
             "weight": (1 + 0.1 * torch.randn(case["width"], device=DEV, generator=g)).to(dt)}
        s["residual"] = _hidden(g, case["rows"], case["width"], dt, 2.0) if case["residual"] else None
    elif op == "norm_bwd":
        dt = DTYPES[case["dtype"]]
        h = _hidden(g, case["rows"], case["width"], dt)
        s = {"h": h, "rstd": torch.rsqrt(h.float().square().mean(1) + EPS),
             "weight": (1 + 0.1 * torch.randn(case["width"], device=DEV, generator=g)).to(dt),
             "dy": _hidden(g, case["rows"], case["width"], dt, 0.1),
             "dsum": _hidden(g, case["rows"], case["width"], dt, 0.1) if case["dsum"] else None}
    elif op == "quant":
        s = {"x": _hidden(g, case["rows"], case["cols"], DTYPES[case["dtype"]])}
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // case["b_rows"])
        s = {"a": _e4m3(g, m, k), "b": _e4m3(g, n, k),
             "a_scale": torch.rand(m, kb, device=DEV, generator=g).add_(0.5).mul_(1 / 110.0),
             "b_scale": torch.rand(nb, kb, device=DEV, generator=g).add_(0.5).mul_(1 / (110.0 * math.sqrt(k)))}
    else:
        dt, sizes = DTYPES[case["dtype"]], _sizes(case)
        total = _flat_size(sizes)
        used = torch.zeros(total, device=DEV)  # what lies between two tensors stays 0
        torch._foreach_add_(_views(used, sizes), 1.0)
        w = torch.randn(total, device=DEV, generator=g).mul_(0.05).mul_(used)
        grad = torch.randn(total, device=DEV, generator=g).mul_(1e-3).mul_(used).to(dt)
        m = torch.randn(total, device=DEV, generator=g).mul_(3e-4).mul_(used)
        v = torch.rand(total, device=DEV, generator=g).add_(0.05).mul_(1e-6).mul_(used)
        # a trainer's flat buffers, and the tensors in them
        s = {"flat": {"params": w.to(dt), "m": m, "v": v}, "grad": grad, "sizes": sizes, "table": None,
             "grads": _views(grad, sizes)}
        if case["dtype"] != "f32":
            s["flat"]["masters"] = w
        if case["state"] == "e4m3":
            s["flat"]["m"], s["flat"]["m_scale"] = _pack(m)
            s["flat"]["v"], s["flat"]["v_scale"] = _pack(v.sqrt(), True)
    return {**case, **s}


# ---------------------------------------------------------------- plain forms


def _scales(amax, top):
    """A block's scale; 1 where the block is held as zeros."""
    return torch.where(amax < TINY, torch.ones_like(amax), amax / top)


def _blocks(y, dim):
    """y with its `dim` split into blocks of 128 (padded with zeros at the end)."""
    n = y.shape[dim]
    pad = -n % BLOCK
    if pad:
        y = torch.nn.functional.pad(y, (0, pad) if dim == 1 else (0, 0, 0, pad))
    return y.unflatten(dim, (-1, BLOCK))


def _to_e4m3(y):
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quantise_rows(y):
    """e4m3 of y [R, C] with a scale for each 128 columns."""
    r, c = y.shape
    b = _blocks(y, 1)
    scale = _scales(b.abs().amax(2), E4M3_MAX)
    return _to_e4m3((b / scale[:, :, None]).flatten(1)[:, :c]), scale


def _pack(p, root=False):
    """A flat state in 8 bits, a scale for each 128 values; a root that is not 0 is never held as 0."""
    n = p.numel()
    b = _blocks(p.reshape(1, n), 1)[0]
    scale = _scales(b.abs().amax(1), E4M3_MAX)
    t = b / scale[:, None]
    if root:
        t = torch.where(t > 0, t.clamp_min(2.0 ** -9), t)
    return _to_e4m3(t.flatten()[:n]), scale


def _unpack(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK)[:q.numel()]


def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None] * s["weight"].float()
    out = {}
    if s["out"] == "i8":
        scale = _scales(y.abs().amax(1), 127.0)
        out["y"] = (torch.round(y / scale[:, None]) * scale[:, None]).to(torch.bfloat16)
    elif s["out"] == "e4m3":
        out["y"], out["scale"] = _quantise_rows(y)
    else:
        out["y"] = y.to(s["x"].dtype)
    if s["residual"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    if s["rstd"]:
        out["rstd"] = rstd
    return out


def _norm_bwd(s):
    dy, xh = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    gw = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (gw - xh * (gw * xh).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xh).sum(0)}


def _quant(s):
    x = s["x"].float()
    r, c = x.shape
    if s["block_rows"] == 1:
        q, scale = _quantise_rows(x)
        out = {"q": q, "scale": scale}
        if s["both"]:
            out["qt"], out["scale_t"] = _quantise_rows(x.t().contiguous())
        return out
    b = _blocks(_blocks(x, 1).flatten(1), 0)                      # [R/128, 128, C padded]
    b = b.unflatten(2, (-1, BLOCK))                               # [R/128, 128, C/128, 128]
    scale = _scales(b.abs().amax((1, 3)), E4M3_MAX)
    q = _to_e4m3((b / scale[:, None, :, None]).flatten(2).flatten(0, 1)[:r, :c])
    out = {"q": q, "scale": scale}
    if s["both"]:
        out["qt"], out["scale_t"] = q.t().contiguous(), scale.t().contiguous()
    return out


def _gemm(s):
    k = s["k"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    b_scale = s["b_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    if s["b_rows"] > 1:
        b_scale = b_scale.repeat_interleave(s["b_rows"], 0)[:s["n"]]
    return {"c": (a @ (s["b"].float() * b_scale).t()).to(DTYPES[s["out"]])}


def _adamw(s):
    f = s["flat"]
    packed = s["state"] == "e4m3"
    g = s["grad"].float()
    p = f.get("masters", f["params"])
    m = _unpack(f["m"], f["m_scale"]) if packed else f["m"]
    v = _unpack(f["v"], f["v_scale"]).square_() if packed else f["v"]
    m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    root = v.sqrt()
    if packed:
        f["m"], f["m_scale"] = _pack(m)
        f["v"], f["v_scale"] = _pack(root, True)
    root = root.div_(math.sqrt(1 - BETA2 ** STEP)).add_(ADAM_EPS)
    p.mul_(1 - LR * DECAY).addcdiv_(m, root, value=-LR / (1 - BETA1 ** STEP))
    if p is not f["params"]:
        f["params"].copy_(p)
    return dict(f)


PLAIN = {"norm": _norm, "norm_bwd": _norm_bwd, "quant": _quant, "gemm": _gemm, "adamw": _adamw}


# ---------------------------------------------------------------- the library's calls


def _own_norm(bd, s):
    kind = s["x"].dtype if s["out"] == "same" else DTYPES[s["out"]]
    y, scale, h, rstd = bd.maxsim_rmsnorm_fwd(s["x"], s["weight"], EPS, residual=s["residual"], out_dtype=kind,
                                              with_rstd=s["rstd"])
    out = {"y": y}
    if s["out"] == "i8":
        out["y"] = torch.mul(y, scale[:, None], out=torch.empty(y.shape, dtype=torch.bfloat16, device=y.device))
    elif scale is not None:
        out["scale"] = scale
    if h is not None:
        out["sum"] = h
    if rstd is not None:
        out["rstd"] = rstd
    return out


def _own_norm_bwd(bd, s):
    dx, dw = bd.maxsim_rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["weight"], dsum=s["dsum"])
    return {"dx": dx, "dweight": dw}


def _own_quant(bd, s):
    q, scale, qt, scale_t = bd.maxsim_quant_fp8(s["x"], block_rows=s["block_rows"], transposed=s["both"])
    out = {"q": q, "scale": scale}
    if s["both"]:
        out["qt"], out["scale_t"] = qt, scale_t
    return out


def _own_gemm(bd, s):
    return {"c": bd.maxsim_gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DTYPES[s["out"]])}


def _own_adamw(bd, s):
    f = s["flat"]
    if s["table"] is None:  # the optimiser's own table of its tensors, made with it
        part = lambda name, per=1: _views(f[name], s["sizes"], per) if name in f else None  # noqa: E731
        s["table"] = bd.AdamWTensors(part("params"), part("m"), part("v"), masters=part("masters"),
                                     m_scales=part("m_scale", BLOCK), v_scales=part("v_scale", BLOCK))
    bd.maxsim_adamw(s["table"], s["grads"], STEP, LR, BETA1, BETA2, ADAM_EPS, DECAY)
    return dict(f)


OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "quant": _own_quant, "gemm": _own_gemm, "adamw": _own_adamw}


def run(state):
    if own:
        from late_interaction_retrieval_amd import binding
        return OWN[state["op"]](binding, state)
    return PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    size = {"f16": 2, "bf16": 2, "f32": 4, "i8": 1, "e4m3": 1}
    if op in ("norm", "norm_bwd", "quant"):
        rows, width, e = case["rows"], case.get("width", case.get("cols")), size[case["dtype"]]
    if op == "norm":
        o = e if case["out"] == "same" else 1
        nbytes = rows * width * (e + o + (2 * e if case["residual"] else 0)) + width * e
        nbytes += 4 * rows * (-(-width // BLOCK) if case["out"] == "e4m3" else 1 if case["out"] == "i8" else 0)
        return {"bytes": nbytes + (4 * rows if case["rstd"] else 0), "flops": 6 * rows * width}
    if op == "norm_bwd":
        return {"bytes": rows * width * e * (4 if case["dsum"] else 3) + 4 * rows + width * (e + 4),
                "flops": 10 * rows * width}
    if op == "quant":
        both = 2 if case["both"] else 1
        scales = -(-rows // case["block_rows"]) * -(-width // BLOCK)
        return {"bytes": rows * width * (e + both) + 4 * both * scales, "flops": 3 * both * rows * width}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": (m + n) * k + 4 * kb * (m + -(-n // case["b_rows"])) + m * n * size[case["out"]],
                "flops": 2 * m * n * k}
    total, e = sum(_sizes(case)), size[case["dtype"]]
    each = 2 * e + e + (8 if case["dtype"] != "f32" else 0) + (16 if case["state"] == "f32" else 4 + 16 / BLOCK)
    if case["dtype"] != "f32":
        each -= e  # a 16-bit weight is written from its master, not read
    return {"bytes": total * each, "flops": 15 * total}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_e4m3(t):
    """t as e4m3 holds it, in 64 bits: 4 significant bits down to 2^-6, nearest, ties to even."""
    _, e = torch.frexp(t)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(t / step) * step


def _exact_blocks(y, br, bc):
    """(values in e4m3, scales) of y [R, C] in blocks of br x bc."""
    r, c = y.shape
    full = y.new_zeros(-(-r // br) * br, -(-c // bc) * bc)
    full[:r, :c] = y
    cut = full.reshape(full.shape[0] // br, br, full.shape[1] // bc, bc)
    top = cut.abs().amax(dim=(1, 3))
    scale = torch.where(top < TINY, 1.0, top / E4M3_MAX)
    return _exact_e4m3(cut / scale[:, None, :, None]).reshape(full.shape)[:r, :c], scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        rstd = (h.pow(2).sum(1) / case["width"] + EPS) ** -0.5
        y = s["weight"].double() * (rstd.unsqueeze(1) * h)
        out = {"y": y}
        if case["out"] == "i8":
            scale = y.abs().max(1, keepdim=True).values / 127
            out["y"] = torch.round(y / scale) * scale
        elif case["out"] == "e4m3":
            out["y"], out["scale"] = _exact_blocks(y, 1, BLOCK)
        if s["residual"] is not None:
            out["sum"] = h
        if case["rstd"]:
            out["rstd"] = rstd
        return out
    if op == "norm_bwd":
        h, r, dy = s["h"].double(), s["rstd"].double().unsqueeze(1), s["dy"].double()
        u = dy * s["weight"].double()
        inner = (u * h).sum(1, keepdim=True)
        dx = r * u - h * r.pow(3) * inner / case["width"]
        return {"dx": dx + (0 if s["dsum"] is None else s["dsum"].double()),
                "dweight": torch.matmul((h * dy).t(), r).squeeze(1)}
    if op == "quant":
        x, br = s["x"].double(), case["block_rows"]
        out = {}
        out["q"], out["scale"] = _exact_blocks(x, br, BLOCK)
        if case["both"]:
            out["qt"], out["scale_t"] = _exact_blocks(x.t(), br, BLOCK)
        return out
    if op == "gemm":
        c = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        width = 2048
        for at in range(0, case["k"], width):  # some blocks of k at a time
            k = torch.arange(at, min(case["k"], at + width), device=DEV)
            rows = torch.arange(case["n"], device=DEV) // case["b_rows"]
            a = s["a"][:, k[0]:k[-1] + 1].double() * s["a_scale"].double()[:, k // BLOCK]
            b = s["b"][:, k[0]:k[-1] + 1].double() * s["b_scale"].double()[rows][:, k // BLOCK]
            c += torch.matmul(a, b.t().contiguous())
        return {"c": c}
    f = s["flat"]
    packed = case["state"] == "e4m3"
    p, g = f.get("masters", f["params"]).double(), s["grad"].double()
    m, v = f["m"].double(), f["v"].double()
    if packed:
        m = (m.view(-1, BLOCK) * f["m_scale"].double().unsqueeze(1)).flatten()
        v = (v.view(-1, BLOCK) * f["v_scale"].double().unsqueeze(1)).flatten() ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    mh, vh = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    p = p - LR * (DECAY * p + mh / (vh ** 0.5 + ADAM_EPS))
    out = {"params": p, "m": m, "v": v}
    if "masters" in f:
        out["masters"] = p
    if packed:
        for name, t in (("m", m), ("v", v.sqrt())):
            q, scale = _exact_blocks(t.unsqueeze(0), 1, BLOCK)
            out[name], out[name + "_scale"] = q[0], scale[0]
    return out
