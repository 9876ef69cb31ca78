"""The operators of the encoder's attention layer and of the loss that trains it, case by case: rotary positions,
attention with a sliding window and first tokens that stay visible (forward, backward, single tokens against a cache),
and distillation from a teacher's top scores (forward and backward).

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
BASE = 10000.0


def listed():
    return [
        # the next token of 8 running sequences, queries and keys of 16 + 4 heads: the smallest call, latency alone
        {"name": "rope_next_token", "op": "rope", "batch": 8, "length": 1, "heads": 20, "width": 64, "rotary": 64,
         "layout": "half", "dtype": "f16", "stretch": 1.0, "positions": "offsets", "far": 32768, "inverse": False},
        # a batch of 32 documents of 1024 tokens, queries and keys of one projection, frequencies stretched for long contexts
        {"name": "rope_documents", "op": "rope", "batch": 32, "length": 1024, "heads": 20, "width": 128, "rotary": 128,
         "layout": "interleaved", "dtype": "bf16", "stretch": 4.0, "positions": "index", "far": 1024, "inverse": False},
        # the gradient of an odd number of packed tokens at far positions, part of an odd head, fp32
        {"name": "rope_backward_odd", "op": "rope", "batch": 1, "length": 5003, "heads": 7, "width": 80, "rotary": 48,
         "layout": "half", "dtype": "f32", "stretch": 8.0, "positions": "given", "far": 2000000, "inverse": True},
        # one query's 32 tokens, every token sees every other: latency
        {"name": "attn_query", "op": "attn", "packed": False, "batch": 1, "lq": 32, "lk": 32, "ragged": 0.0, "hq": 12,
         "hk": 12, "width": 64, "dtype": "f16", "left": -1, "right": -1, "sinks": 0, "train": False, "shape_seed": 1},
        # documents of 32 to 1024 tokens, packed, in a layer that sees 128 tokens to each side and the first one
        {"name": "attn_documents", "op": "attn", "packed": True, "batch": 64, "lq": 1024, "lk": 1024, "ragged": 0.97,
         "hq": 16, "hk": 16, "width": 64, "dtype": "bf16", "left": 128, "right": 128, "sinks": 1, "train": False,
         "shape_seed": 2},
        # a long text into a decoder's cache: causal, 2048 tokens back and the first 4
        {"name": "attn_long", "op": "attn", "packed": False, "batch": 1, "lq": 8192, "lk": 8192, "ragged": 0.0, "hq": 32,
         "hk": 8, "width": 128, "dtype": "bf16", "left": 2047, "right": 0, "sinks": 4, "train": False, "shape_seed": 3},
        # the next token of 16 sequences against caches of up to 32768 tokens: the cache's bytes
        {"name": "attn_next_token", "op": "attn", "packed": False, "batch": 16, "lq": 1, "lk": 32768, "ragged": 0.75,
         "hq": 32, "hk": 8, "width": 128, "dtype": "bf16", "left": -1, "right": 0, "sinks": 0, "train": False,
         "shape_seed": 4},
        # a small training batch of odd lengths (none and one among them), three heads to a key head of 80
        {"name": "attn_train_odd", "op": "attn", "packed": True, "batch": 9, "lq": 601, "lk": 601, "ragged": 1.0, "hq": 6,
         "hk": 2, "width": 80, "dtype": "f16", "left": 100, "right": 0, "sinks": 3, "train": True, "shape_seed": 5},
        # a training step's documents in a layer that sees everything, padded to 1024 tokens
        {"name": "attn_train_documents", "op": "attn", "packed": False, "batch": 16, "lq": 1024, "lk": 1024, "ragged": 0.3,
         "hq": 16, "hk": 4, "width": 128, "dtype": "bf16", "left": -1, "right": -1, "sinks": 0, "train": True,
         "shape_seed": 6},
        # 64 queries' scores of the 64 documents in their batch: latency
        {"name": "distill_in_batch", "op": "distill", "rows": 64, "cols": 64, "top": 16, "dtype": "f32",
         "temperature": 1.0},
        # a few queries' scores of a whole corpus, the teacher's best 100 of each
        {"name": "distill_corpus", "op": "distill", "rows": 32, "cols": 200003, "top": 100, "dtype": "f32",
         "temperature": 2.0},
        # a training step's tokens over a vocabulary
        {"name": "distill_vocabulary", "op": "distill", "rows": 8192, "cols": 32768, "top": 64, "dtype": "bf16",
         "temperature": 2.0},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "attn", "distill"])
    if op == "rope":
        width = rng.choice([64, 128, 2 * _spread(rng, 16, 64), _spread(rng, 32, 128)])
        heads = _spread(rng, 1, 40)
        batch = _spread(rng, 1, 64)
        length = _spread(rng, 1, max(1, (16384 * 20 * 128) // (batch * heads * width)))
        return {"op": op, "batch": batch, "length": min(length, 32768), "heads": heads, "width": width,
                "rotary": rng.choice([width // 2 * 2, width // 4 * 2, 2 * rng.randint(1, width // 2)]),
                "layout": rng.choice(["half", "interleaved"]), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "stretch": rng.choice([1.0, 2.0, 8.0]), "positions": rng.choice(["offsets", "index", "given"]),
                "far": _spread(rng, 64, 2000000), "inverse": rng.random() < 0.4}
    if op == "distill":
        cols = _spread(rng, 8, 262144)
        return {"op": op, "rows": _spread(rng, 1, max(1, min(16384, (1 << 27) // cols))), "cols": cols,
                "top": min(cols, _spread(rng, 1, 256)), "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
                "temperature": rng.choice([1.0, 2.0, 0.5])}
    hk = _spread(rng, 1, 16)
    hq = hk * rng.choice([1, 1, 2, 3, 4, 8])
    width = rng.choice([64, 64, 128, 128, 8 * rng.randint(2, 16)])
    kind = rng.choice(["encode", "encode", "next", "append", "train", "train"])
    batch = _spread(rng, 1, 64)
    # values of the plain form's largest tensor (the score of every pair), and of the keys
    most = 1 << 27 if kind == "train" else 1 << 29
    if kind in ("next", "append"):
        lk = _spread(rng, 64, max(65, min(32768, (1 << 28) // (batch * hk * width))))
        lq = 1 if kind == "next" else min(lk, _spread(rng, 2, max(2, min(512, most // (batch * hq * lk)))))
    else:
        lk = lq = _spread(rng, 16, max(17, min(8192, int(math.sqrt(most / (batch * hq))))))
    left = rng.choice([-1, _spread(rng, 1, 2048), _spread(rng, 1, 256)])
    right = 0 if kind in ("next", "append") else rng.choice([0, 0, -1, left])
    return {"op": op, "packed": kind in ("encode", "train") and rng.random() < 0.6, "batch": batch, "lq": lq, "lk": lk,
            "ragged": rng.choice([0.0, 0.5, 0.9, 1.0]), "hq": hq, "hk": hk, "width": width,
            "dtype": rng.choice(["bf16", "bf16", "f16"]), "left": left, "right": right,
            "sinks": rng.choice([0, 1, 4]) if left >= 0 else 0, "train": kind == "train",
            "shape_seed": rng.randrange(1 << 30)}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _lengths(case):
    """(queries, keys) of each sequence: the first has the most, the others some of up to `ragged` of it fewer."""
    r = random.Random(case["shape_seed"])
    keep = [1.0] + [1.0 - case["ragged"] * r.random() ** 0.7 for _ in range(case["batch"] - 1)]
    lk = [max(int(case["lk"] * f + 0.5), min(1, case["lk"]) if case["ragged"] < 1 else 0) for f in keep]
    if case["ragged"] >= 1 and case["batch"] > 4:
        lk[2], lk[3] = 0, 1  # a text of nothing, and one of a single token
    if case["lq"] == case["lk"]:
        return list(lk), lk
    return [min(case["lq"], k) for k in lk], lk


def _starts(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _frequencies(rotary, stretch):
    """Angles a position, in 64 bits; stretched contexts divide the slow ones by `stretch` and leave the fast ones."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device=DEV)
    f = BASE ** (-2 * i / rotary)
    if stretch == 1.0:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)  # of each pair over the length that the weights were trained on
    slow = ((32 - turns) / 31).clamp(0, 1)
    return f * (1 - slow + slow / stretch), 1 + 0.1 * math.log(stretch)


def prepare(case, seed):
    g = _generator(seed)
    randn = lambda *shape: torch.randn(*shape, device=DEV, generator=g)  # noqa: E731
    s = {}
    if case["op"] == "rope":
        dt = DTYPES[case["dtype"]]
        lead = (case["length"],) if case["positions"] == "given" and case["batch"] == 1 else (case["batch"], case["length"])
        s["x"] = randn(*lead, case["heads"], case["width"]).to(dt)
        s["inv_freq"], s["scale"] = _frequencies(case["rotary"], case["stretch"])
        integers = lambda *shape: torch.randint(0, case["far"], shape, device=DEV, generator=g, dtype=torch.int32)  # noqa: E731
        s["offsets"] = integers(case["batch"]) if case["positions"] == "offsets" else None
        s["given"] = integers(*lead) if case["positions"] == "given" else None
    elif case["op"] == "attn":
        dt = DTYPES[case["dtype"]]
        lq, lk = _lengths(case)
        D, hq, hk = case["width"], case["hq"], case["hk"]
        if case["packed"]:
            q, k = (max(1, sum(lq)),), (max(1, sum(lk)),)
            s["cu_q"] = s["cu_k"] = _starts(lk)
            s["q_lens"] = s["k_lens"] = None
        else:
            q, k = (case["batch"], case["lq"]), (case["batch"], case["lk"])
            whole = case["ragged"] == 0
            s["cu_q"] = s["cu_k"] = None
            ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
            s["q_lens"] = None if whole or min(lq) == case["lq"] else ints(lq)
            s["k_lens"] = None if whole else ints(lk)
        s["q"] = (1.5 * randn(*q, hq, D)).to(dt)
        s["k"] = randn(*k, hk, D).to(dt)
        s["v"] = randn(*k, hk, D).to(dt)
        s["dout"] = randn(*q, hq, D).to(dt) if case["train"] else None
    else:
        n, v, k = case["rows"], case["cols"], case["top"]
        s["scores"] = (3.0 * randn(n, v)).to(DTYPES[case["dtype"]])
        # what the teacher likes best: k different columns of each row, one in each k-th part of it
        at = torch.arange(k, device=DEV) * v // k
        wide = (torch.arange(1, k + 1, device=DEV) * v // k) - at
        s["index"] = (at + (torch.rand(n, k, device=DEV, generator=g) * wide).long().clamp_max(wide - 1)).to(torch.int32)
        s["teacher"] = 3.0 * randn(n, k).abs()
        s["dloss"] = torch.rand(n, device=DEV, generator=g).add_(0.5).div_(n)
    return {**case, **s}


# ---------------------------------------------------------------- plain forms


def _rope(s):
    x = s["x"].float()
    L, half = x.shape[-3], s["rotary"] // 2
    if s["given"] is not None:
        at = s["given"].double()
    else:
        at = torch.arange(L, dtype=torch.float64, device=DEV)
        at = at.expand(s["batch"], L) if s["offsets"] is None else at + s["offsets"].double()[:, None]
    angle = at[..., None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["scale"]).float()[..., None, :] for f in (torch.cos, torch.sin))
    if s["inverse"]:
        sin = -sin
    r = x[..., :2 * half]
    if s["layout"] == "half":
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return {"y": torch.cat([r, x[..., 2 * half:]], -1).to(s["x"].dtype)}


def _dense(t, cu, lens, L, heads):
    """t in 32 bits as [batch, heads, rows, width] with the rows of `heads` query heads after each other; zeros past a
    sequence's end; and the lengths."""
    if cu is not None:
        at = torch.arange(L, device=DEV)
        rows = cu[:-1, None].long() + at
        n = (cu[1:] - cu[:-1]).long()
        t = t[rows.clamp_max(t.shape[0] - 1)]
    else:
        n = torch.full((t.shape[0],), L, device=DEV) if lens is None else lens.long()
        at = torch.arange(L, device=DEV)
    t = torch.where((at < n[:, None])[:, :, None, None], t, torch.zeros((), dtype=t.dtype, device=DEV)).float()
    B, _, H, D = t.shape
    return t.unflatten(2, (H // heads, heads)).permute(0, 2, 3, 1, 4).reshape(B, H // heads, heads * L, D), n


def _undense(t, like, cu, L, heads):
    """_dense()'s rows back in the layout of `like`."""
    B, H, _, D = t.shape
    t = t.reshape(B, H, heads, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, H * heads, D)
    if cu is not None:
        rows = torch.arange(like.shape[0], device=DEV, dtype=torch.int32)
        b = (torch.searchsorted(cu, rows, right=True) - 1).clamp_max(B - 1)
        t = t[b, (rows - cu[b]).long().clamp_max(L - 1)]
    return t.to(like.dtype)


def _attn(s):
    group, Lq, Lk = s["hq"] // s["hk"], s["lq"], s["lk"]
    q, nq = _dense(s["q"], s["cu_q"], s["q_lens"], Lq, group)
    k, nk = _dense(s["k"], s["cu_k"], s["k_lens"], Lk, 1)
    v, _ = _dense(s["v"], s["cu_k"], s["k_lens"], Lk, 1)
    i, j = torch.arange(Lq, device=DEV)[None, :, None], torch.arange(Lk, device=DEV)
    p = i + (nk - nq)[:, None, None]
    seen = (i < nq[:, None, None]) & (j < nk[:, None, None])
    if s["right"] >= 0:
        seen = seen & (j <= p + s["right"])
    if s["left"] >= 0:
        seen = seen & ((j >= p - s["left"]) | (j < s["sinks"]))
    hidden = ~seen.repeat(1, group, 1)[:, None]
    scale = 1 / math.sqrt(s["width"])
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = e.sum(-1, keepdim=True)
    part = e.div_(torch.where(total > 0, total, 1.0))
    out = {"out": _undense(torch.matmul(part, v), s["q"], s["cu_q"], Lq, group)}
    if not s["train"]:
        return out
    do, _ = _dense(s["dout"], s["cu_q"], s["q_lens"], Lq, group)
    dp = torch.matmul(do, v.transpose(2, 3).contiguous())
    out["dv"] = _undense(torch.matmul(part.transpose(2, 3).contiguous(), do), s["v"], s["cu_k"], Lk, 1)
    dp.sub_((part * dp).sum(-1, keepdim=True)).mul_(part).mul_(scale)
    out["dq"] = _undense(torch.matmul(dp, k), s["q"], s["cu_q"], Lq, group)
    out["dk"] = _undense(torch.matmul(dp.transpose(2, 3).contiguous(), q), s["k"], s["cu_k"], Lk, 1)
    return out


def _distill(s):
    t = s["temperature"]
    z = s["scores"].float() / t
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    index = s["index"].long()
    want = s["teacher"] / t
    want = want - want.amax(1, keepdim=True)
    log_q = want - want.exp().sum(1, keepdim=True).log()
    q = log_q.exp()
    loss = t * t * (q * (log_q - (z.gather(1, index) - top - total.log()))).sum(1)
    dz = (e / total).scatter_add_(1, index, -q)
    return {"loss": loss, "dscores": (dz * (t * s["dloss"])[:, None]).to(s["scores"].dtype)}


PLAIN = {"rope": _rope, "attn": _attn, "distill": _distill}


# ---------------------------------------------------------------- the library's calls


def _own_rope(bd, s):
    return {"y": bd.maxsim_rope(s["x"], s["inv_freq"], positions=s["given"], offsets=s["offsets"], layout=s["layout"],
                                scale=s["scale"], inverse=s["inverse"])}


def _own_attn(bd, s):
    how = dict(window=(s["left"], s["right"]), sinks=s["sinks"])
    if s["cu_q"] is not None:
        how.update(cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=s["lq"], max_k=s["lk"])
    else:
        how.update(q_lens=s["q_lens"], k_lens=s["k_lens"])
    out, lse = bd.maxsim_attn_fwd(s["q"], s["k"], s["v"], with_lse=s["train"], **how)
    if not s["train"]:
        return {"out": out}
    dq, dk, dv = bd.maxsim_attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **how)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _own_distill(bd, s):
    loss, lse = bd.maxsim_distill_fwd(s["scores"], s["index"], s["teacher"], temperature=s["temperature"])
    return {"loss": loss, "dscores": bd.maxsim_distill_bwd(s["dloss"], s["scores"], lse, s["index"], s["teacher"],
                                                           temperature=s["temperature"])}


OWN = {"rope": _own_rope, "attn": _own_attn, "distill": _own_distill}


def run(state):
    if own:
        from late_interaction_retrieval_amd import binding
        return OWN[state["op"]](binding, state)
    return PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without


def _pairs(case):
    """(query, key) pairs of one head that see each other, and the keys that any query sees."""
    pairs = keys = 0
    for nq, nk in zip(*_lengths(case)):
        p = torch.arange(nq) + nk - nq
        hi = torch.full((nq,), nk) if case["right"] < 0 else (p + case["right"] + 1).clamp(0, nk)
        lo = torch.zeros(nq, dtype=torch.long) if case["left"] < 0 else (p - case["left"]).clamp(0, nk)
        first = torch.minimum(torch.full((nq,), case["sinks"]), torch.minimum(lo, hi))
        seen = (hi - lo).clamp_min(0) + first
        pairs += int(seen.sum())
        if nq:
            keys += max(0, int(hi.max()) - int(lo.min())) + min(int(lo.min()), case["sinks"])
    return pairs, keys


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "rope":
        tokens = case["batch"] * case["length"]
        at = tokens if case["positions"] == "given" else case["batch"] if case["positions"] == "offsets" else 0
        return {"bytes": 2 * tokens * case["heads"] * case["width"] * e + 4 * at + 4 * case["rotary"],
                "flops": 3 * tokens * case["heads"] * case["rotary"]}
    if case["op"] == "distill":
        n, v, k = case["rows"], case["cols"], case["top"]
        return {"bytes": 2 * n * v * e + 8 * n * k + 8 * n, "flops": 8 * n * v}
    pairs, keys = _pairs(case)
    rows, kv = sum(_lengths(case)[0]) * case["hq"] * case["width"] * e, keys * case["hk"] * case["width"] * e
    if not case["train"]:
        return {"bytes": 2 * rows + 2 * kv, "flops": 4 * pairs * case["hq"] * case["width"]}
    return {"bytes": 4 * rows + 4 * kv, "flops": 14 * pairs * case["hq"] * case["width"]}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_rope(s):
    x, R = s["x"].double(), s["rotary"]
    flat = x.reshape(-1, s["heads"], s["width"])
    token = torch.arange(flat.shape[0], device=DEV)
    if s["given"] is not None:
        at = s["given"].reshape(-1).long()
    else:
        at = token % s["length"]
        if s["offsets"] is not None:
            at = at + s["offsets"].long()[token // s["length"]]
    turn = torch.polar(torch.full((R // 2,), s["scale"], dtype=torch.float64, device=DEV), torch.zeros_like(s["inv_freq"]))
    angle = torch.outer(at.double(), s["inv_freq"])
    turn = turn * torch.complex(torch.cos(angle), torch.sin(angle) * (-1 if s["inverse"] else 1))
    pairs = flat[..., :R]
    pairs = pairs.unflatten(-1, (2, R // 2)).transpose(-1, -2) if s["layout"] == "half" else pairs.unflatten(-1, (R // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    z = z.transpose(-1, -2).flatten(-2) if s["layout"] == "half" else z.flatten(-2)
    return {"y": torch.cat([z, flat[..., R:]], -1).reshape(x.shape)}


def _exact_attn(s):
    lens = list(zip(*_lengths(s)))
    names = ["q", "k", "v"] + (["dout"] if s["train"] else [])
    out = {n: torch.zeros_like(s[m], dtype=torch.float64)
           for n, m in [("out", "q")] + ([("dq", "q"), ("dk", "k"), ("dv", "v")] if s["train"] else [])}
    group = s["hq"] // s["hk"]
    qa = ka = 0
    for b, (nq, nk) in enumerate(lens):
        if s["packed"]:
            rows = {"q": slice(qa, qa + nq), "k": slice(ka, ka + nk)}
            qa, ka = qa + nq, ka + nk
        else:
            rows = {"q": (b, slice(0, nq)), "k": (b, slice(0, nk))}
        rows.update(v=rows["k"], dout=rows["q"], out=rows["q"], dq=rows["q"], dk=rows["k"], dv=rows["k"])
        if nq == 0 or nk == 0:
            continue
        delta = torch.arange(nk, device=DEV) - (torch.arange(nq, device=DEV)[:, None] + (nk - nq))  # key - position
        bias = torch.zeros(nq, nk, dtype=torch.float64, device=DEV)
        if s["right"] >= 0:
            bias[delta > s["right"]] = -math.inf
        if s["left"] >= 0:
            far = delta < -s["left"]
            far[:, :s["sinks"]] = False
            bias[far] = -math.inf
        blind = torch.isinf(bias).all(1)
        for h in range(s["hq"]):
            x = {n: s[n][rows[n]][:, h if n in ("q", "dout") else h // group].double() for n in names}
            for n in ("q", "k", "v"):
                x[n].requires_grad_(s["train"])
            logits = torch.matmul(x["q"], x["k"].t()) / s["width"] ** 0.5 + bias
            o = torch.matmul(torch.softmax(logits.masked_fill(blind[:, None], 0.0), 1), x["v"])
            o = o.masked_fill(blind[:, None], 0.0)
            out["out"][rows["out"]][:, h] = o.detach()
            if s["train"]:
                dq, dk, dv = torch.autograd.grad(o, [x["q"], x["k"], x["v"]], x["dout"])
                out["dq"][rows["dq"]][:, h] = dq
                out["dk"][rows["dk"]][:, h // group] += dk
                out["dv"][rows["dv"]][:, h // group] += dv
    return out


def _exact_distill(s):
    t, n = s["temperature"], s["rows"]
    loss = torch.empty(n, dtype=torch.float64, device=DEV)
    grad = torch.empty(n, s["cols"], dtype=torch.float64, device=DEV)
    step = max(1, (1 << 25) // s["cols"])
    for at in range(0, n, step):
        z = s["scores"][at:at + step].double().requires_grad_()
        log_p = torch.log_softmax(z / t, 1).gather(1, s["index"][at:at + step].long())
        log_q = torch.log_softmax(s["teacher"][at:at + step].double() / t, 1)
        rows = t ** 2 * (torch.exp(log_q) * (log_q - log_p)).sum(1)
        loss[at:at + step] = rows.detach()
        grad[at:at + step] = torch.autograd.grad(rows, z, s["dloss"][at:at + step].double())[0]
    return {"loss": loss, "dscores": grad}


def exact(case, seed):
    if case["op"] == "attn":
        lq, lk = _lengths(case)
        heads = case["batch"] * case["hq"]
        if heads > 4096 or sum(a * b for a, b in zip(lq, lk)) * case["hq"] > 1 << 33:
            return None  # a pass of each head alone: too many of them
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "distill": _exact_distill}[case["op"]](s)
