"""The operators of a 4-bit decoder layer with a sliding window, as cases to be measured.

A decoder layer whose linears are held in 4 bits, and whose attention looks at
a window and a few first positions, runs next to the 8-bit calls: the
quantisation of activations to microscaled 4-bit numbers, their product with a
weight of the same format, the norm and rotation of each head's queries and
keys, and the attention over the paged 8-bit cache with a window and sinks.
Each case is one call of one of them (quant: there and back).

    quant    blocks of 32 values along a row, with one power of two each:
             scale = 2^(floor(log2(max |x|)) - 2), at least 2^-127;
             code = x / scale rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3,
             4, 6 and their negatives, ties to the even code, at most 6;
             a block that holds infinity or NaN reads as NaN throughout
    product  sum over k of a[i][k] b[j][k], a and b the values their codes
             and scales stand for
    linear   the product with the activations quantised first
    rotate   y = x / sqrt(mean(x^2) + eps) * w over a head's elements, then
             each pair (y_i, y_i+r/2), or (y_2i, y_2i+1), of the first r
             turned by the angle position * frequency_i
    attend   softmax(q k^T * D^-1/2) v over the cached positions j <= p of a
             row at position p with j > p - window or j < sinks

Codes are two to a byte, the lower position in the lower half; scales are the
powers' exponents plus 127, a byte each (255: NaN), in rows that begin at a
multiple of 16 bytes.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ---- cases ----

def listed():
    return [
        # the activations of one decode step of 8 requests: latency
        {"name": "quant_decode", "op": "quant", "m": 8, "k": 4096, "dtype": "bf16"},
        # the gated MLP workload's 4096 tokens before the down projection
        {"name": "quant_large", "op": "quant", "m": 4096, "k": 14336, "dtype": "bf16"},
        # the decode workload's up projection for one token: the weight's bytes count
        {"name": "product_decode", "op": "product", "m": 1, "k": 4096, "n": 14336, "out": "bf16"},
        # and for the tokens of a batch of 24 requests
        {"name": "product_batch", "op": "product", "m": 24, "k": 4096, "n": 14336, "out": "bf16"},
        # the prefill workload, 2048 tokens of width 4096
        {"name": "product_prefill", "op": "product", "m": 2048, "k": 4096, "n": 4096, "out": "bf16"},
        # the MLP workload's up projection: the matrix cores count
        {"name": "product_large", "op": "product", "m": 8192, "k": 8192, "n": 28672, "out": "bf16"},
        # a piece of a prompt through a whole linear of odd sizes
        {"name": "linear_odd", "op": "linear", "m": 333, "k": 2720, "n": 1001, "dtype": "f16", "out": "f32"},
        # queries and keys of one new token for each of 64 running requests: latency
        {"name": "rotate_tokens", "op": "rotate", "seqs": 64, "start_lo": 1, "start_hi": 8191, "new_lo": 1, "new_hi": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False, "norm": True, "dtype": "bf16", "lengths": 1},
        # those of five prompts of mixed lengths, half of each head turned
        {"name": "rotate_prompts", "op": "rotate", "seqs": 5, "start_lo": 0, "start_hi": 70000, "new_lo": 700, "new_hi": 2500, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 64, "interleaved": True, "norm": True, "dtype": "bf16", "lengths": 2},
        # the next tokens of 64 requests of mixed lengths, a window of 1024
        {"name": "attend_batch", "op": "attend", "seqs": 64, "new_lo": 1, "new_hi": 1, "len_lo": 1, "len_hi": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "window": 1024, "sinks": 4, "dtype": "bf16", "format": "int8", "lengths": 3},
        # the next tokens of two requests far into long documents, a wide window
        {"name": "attend_long_fp8", "op": "attend", "seqs": 2, "new_lo": 1, "new_hi": 1, "len_lo": 100003, "len_hi": 131071, "heads": 64,
         "kv_heads": 8, "dim": 128, "block": 64, "window": 32768, "sinks": 128, "dtype": "bf16", "format": "fp8", "lengths": 4},
        # a prompt of 4096 tokens, a window of 1024: arithmetic counts
        {"name": "attend_prompt", "op": "attend", "seqs": 1, "new_lo": 4096, "new_hi": 4096, "len_lo": 4096, "len_hi": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "window": 1024, "sinks": 4, "dtype": "bf16", "format": "int8", "lengths": 5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "product", "linear", "rotate", "rotate", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("quant", "product", "linear"):
        m = _log(rng, 1, 8192)
        # a model's width, or any number of whole blocks
        k = rng.choice([512, 1024, 2048, 2560, 4096, 5120, 8192, 14336]) if rng.random() < 0.6 else 32 * _log(rng, 1, 448)
        if op == "quant":
            return {"op": op, "m": m, "k": k, "dtype": rng.choice([dtype, "f32"]) if m * k < 1 << 25 else dtype}
        n = rng.choice([1024, 4096, 6144, 8192, 14336, 28672]) if rng.random() < 0.6 else _log(rng, 16, 28672) | 1
        while m * n * k > 8192 * 8192 * 14336:
            m = (m + 1) // 2
        case = {"op": op, "m": m, "k": k, "n": n, "out": rng.choice(["bf16", "bf16", "f16", "f32"])}
        return case if op == "product" else {**case, "dtype": rng.choice([dtype, "f32"])}
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 7, 8, 16] if kv_heads <= 4 else [1, 2, 4])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 80, 96, 112, 128, 128, 256]), "dtype": dtype,
            "lengths": rng.randrange(1 << 20)}
    if op == "rotate":
        tokens = _log(rng, 1, (12288 * 5120) // ((heads + kv_heads) * case["dim"]))
        seqs = min(tokens, _log(rng, 1, 256))
        most = max(1, tokens // seqs)
        start = rng.choice([0, 1, 5000, 500000])
        return {**case, "dtype": rng.choice([dtype, dtype, "f32"]), "seqs": seqs, "start_lo": min(1, start), "start_hi": start, "new_lo": 1,
                "new_hi": most, "rotary": case["dim"] // rng.choice([1, 1, 2]), "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.7}
    case |= {"block": rng.choice([16, 32, 64, 128]), "format": rng.choice(["int8", "fp8"]), "window": rng.choice([1, 64, 128, 1000, 1024, 4096]),
             "sinks": rng.choice([1, 4, 4, 16, 64, 128, 300])}
    if rng.random() < 0.6:  # single tokens, or a few for each request
        tokens = _log(rng, 64, (230000 * 1024) // (kv_heads * case["dim"]))
        seqs = min(tokens, _log(rng, 1, 64))
        few = rng.choice([1, 1, 1, 4])
        return {**case, "seqs": seqs, "new_lo": few, "new_hi": few, "len_lo": few, "len_hi": max(few, min(131072, tokens // seqs))}
    most = 4096 if heads * case["dim"] <= 4096 else 2048
    new = _log(rng, 17, most)
    seqs = max(1, min(8, most // new))
    return {**case, "seqs": seqs, "new_lo": max(1, new // 2), "new_hi": new, "len_lo": new, "len_hi": max(new, min(4096, 2 * new))}


def _lengths(case):
    """What the case's sequences look like: [(positions before, new positions)] of each, from the case alone."""
    r = random.Random(case["lengths"])
    n = case["seqs"]
    if case["op"] == "rotate":
        return [(r.randint(case["start_lo"], case["start_hi"]), r.randint(case["new_lo"], case["new_hi"])) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    total = [max(x, r.randint(case["len_lo"], case["len_hi"])) for x in new]
    return [(t - x, x) for t, x in zip(total, new)]


def work(case):
    def size(dtype):
        return torch.finfo(DTYPES[dtype]).bits // 8

    if case["op"] == "quant":  # read, written as codes and scales, those read, the values written
        n = case["m"] * case["k"]
        return {"bytes": 2 * n * size(case["dtype"]) + 2 * (n // 2 + n // 32), "flops": 4 * n}
    if case["op"] in ("product", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        a = m * k * size(case["dtype"]) if case["op"] == "linear" else m * (k // 2 + k // 32)
        return {"bytes": a + n * (k // 2 + k // 32) + m * n * size(case["out"]), "flops": 2 * m * n * k}
    tokens = sum(new for _, new in _lengths(case))
    if case["op"] == "rotate":
        n = tokens * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * n * size(case["dtype"]), "flops": (4 * case["norm"] + 3) * n}
    w, s = case["window"], case["sinks"]
    seen = pairs = 0
    for before, new in _lengths(case):
        seen += min(before + new, w + new - 1 + min(s, max(0, before + 1 - w)))
        pairs += sum(min(p + 1, w + min(s, max(0, p + 1 - w))) for p in range(before, before + new))
    return {"bytes": 2 * seen * case["kv_heads"] * case["dim"] + 2 * tokens * case["heads"] * case["dim"] * size(case["dtype"]),
            "flops": 4 * case["dim"] * case["heads"] * pairs}


# ---- the format ----

def _values(q, scale):
    """What codes and scales stand for, in 32 bits."""
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    levels = torch.cat([levels, -levels])
    v = torch.stack([levels[(q & 15).int()], levels[(q >> 4).int()]], -1).flatten(-2)
    s = torch.ldexp(torch.ones((), device=q.device), scale.int() - 127)
    s = torch.where(scale == 255, math.nan, s)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _quantised(x):
    """Codes and scales of x [rows, k]."""
    v = x.float().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1)
    bad = ~v.isfinite().all(-1)
    e = (torch.frexp(top)[1] - 3).clamp_min(-127)  # top = f * 2^e with f from 0.5 up
    e = torch.where(bad | (top == 0), -127, e)
    # in two steps, as 2^127 * 2^3 would not do in one
    u = torch.ldexp(torch.ldexp(v, -(e // 2)[..., None]), -(e - e // 2)[..., None])
    u = torch.where(bad[..., None], 0.0, u)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = ((a / step).round() * step).clamp_max(6)  # ties to even multiples, which are the even codes
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (u.signbit().to(torch.uint8) << 3)).flatten(-2)
    scale = torch.where(bad, 255, e + 127).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _rows_of_scales(scale):
    """The same scales in rows that begin at multiples of 16 bytes."""
    rows, n = scale.shape
    at = torch.zeros(rows, (n + 15) // 16 * 16, dtype=torch.uint8, device=scale.device)
    at[:, :n] = scale
    return at[:, :n]


# ---- inputs ----

def prepare(case, seed):
    dev, g = torch.device("cuda:0"), torch.Generator(device="cuda:0")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    state = {"case": case}
    if case["op"] in ("quant", "product", "linear"):
        m, k = case["m"], case["k"]
        x = randn(m, k)
        x[:, torch.randint(k, (max(1, k // 100),), generator=g, device=dev)] *= 20  # a few large channels
        if case["op"] != "product":
            state["x"] = x.to(DTYPES[case["dtype"]])
        else:
            q, scale = _quantised(x)
            state["a"], state["scale_a"] = q.contiguous(), _rows_of_scales(scale)
        if case["op"] != "quant":
            parts = [_quantised(randn(rows, k) * k ** -0.5) for rows in _pieces(case["n"])]
            state["w"] = torch.cat([q for q, _ in parts])
            state["scale_w"] = _rows_of_scales(torch.cat([s for _, s in parts]))
        return state

    heads, kv, dim, dt = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    new = [n for _, n in lens]
    state |= {"cu": ints([sum(new[:i]) for i in range(len(new) + 1)]), "tokens": sum(new), "most": max(new),
              "start": ints([s for s, _ in lens]), "total": ints([s + n for s, n in lens])}
    if case["op"] == "rotate":
        # queries and keys as slices of one projection's output, as a layer has them
        rows = randn(sum(new), (heads + 2 * kv) * dim).to(dt)
        state["q"] = rows[:, :heads * dim].view(-1, heads, dim)
        state["k"] = rows[:, heads * dim:(heads + kv) * dim].view(-1, kv, dim)
        r = case["rotary"]
        state["freqs"] = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
        state["w"] = [(1 + 0.2 * randn(dim)).to(dt) if case["norm"] else None for _ in range(2)]
        return state

    size, fp8 = case["block"], case["format"] == "fp8"
    each = [(before + n + size - 1) // size for before, n in lens]
    blocks = sum(each)
    # every sequence's blocks lie anywhere in the pool; entries past its end name block 0 and are never read
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), max(each), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(each):
        table[i, :n] = order[at:at + n]
        at += n

    def codes(*shape):
        if fp8:
            return (randn(*shape) * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return (randn(*shape) * 32).clamp_(-127, 127).round_().to(torch.int8)

    def scales():
        return (0.5 + torch.rand(blocks, kv, generator=g, device=dev)) / (110.0 if fp8 else 32.0)

    state["cache"] = (codes(blocks, kv, size, dim), codes(blocks, kv, dim, size), scales(), scales())
    state["table"], state["q"] = table, randn(sum(new), heads, dim).to(dt)
    return state


def _pieces(n):
    """n rows in pieces that are quantised at a time."""
    return [min(4096, n - i) for i in range(0, n, 4096)]


# ---- one pass ----

def run(state):
    case = state["case"]
    if own:
        import w8a8_int8_quantized_qk_amd as qk
        if case["op"] == "quant":
            q, scale = qk.quant_mx4(state["x"])
            return {"values": qk.dequant_mx4(q, scale, DTYPES[case["dtype"]])}
        if case["op"] == "product":
            return {"out": qk.gemm_mx4_scaled(state["a"], state["w"], state["scale_a"], state["scale_w"], out_dtype=DTYPES[case["out"]])}
        if case["op"] == "linear":
            return {"out": qk.linear_mx4(state["x"], state["w"], state["scale_w"], out_dtype=DTYPES[case["out"]])}
        cu = None if state["most"] == 1 else state["cu"]
        if case["op"] == "rotate":
            q, k = qk.norm_rope(state["q"], state["k"], state["start"], state["freqs"], cu, q_weight=state["w"][0], k_weight=state["w"][1],
                                eps=EPS, interleaved=case["interleaved"])
            return {"q": q, "k": k}
        return {"out": qk.kv_attention(state["q"], qk.KVCache(*state["cache"]), state["table"], state["total"], cu,
                                       window=case["window"], sinks=case["sinks"], max_q=state["most"])}
    return {"quant": _quant, "product": _product, "linear": _linear, "rotate": _rotate, "attend": _attend}[case["op"]](state)


def _quant(state):
    return {"values": _values(*_quantised(state["x"])).to(state["x"].dtype)}


def _product(state):
    a, w = _values(state["a"], state["scale_a"]), _values(state["w"], state["scale_w"])
    return {"out": torch.matmul(a, w.t()).to(DTYPES[state["case"]["out"]])}


def _linear(state):
    a, w = _values(*_quantised(state["x"])), _values(state["w"], state["scale_w"])
    return {"out": torch.matmul(a, w.t()).to(DTYPES[state["case"]["out"]])}


def _rotate(state):
    case, cu, r = state["case"], state["cu"].long(), state["case"]["rotary"]
    t = torch.arange(state["tokens"], device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = t - cu[seq] + state["start"].long()[seq]
    angle = pos[:, None, None].double() * state["freqs"]
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for name, w in zip(("q", "k"), state["w"]):
        x = state[name].float()
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.float()
        if case["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out[name] = torch.cat([turned, x[..., r:]], -1).to(state[name].dtype)
    return out


def _held(codes, *at):
    """codes[at] in 32 bits."""
    return codes.view(torch.uint8)[at].view(codes.dtype).float()


def _attend(state):
    kc, vc, ks, vs = state["cache"]
    q, cu, total, case = state["q"], state["cu"].long(), state["total"].long(), state["case"]
    page = state["table"].long()
    seqs, (_, heads, size, dim) = page.shape[0], kc.shape
    length, group, most = page.shape[1] * size, q.shape[1] // heads, state["most"]
    k = _held(kc, page) * ks[page][..., None, None]  # [sequence, block, head, position, dim]
    k = k.permute(0, 2, 4, 1, 3).reshape(seqs * heads, dim, length)
    v = _held(vc, page) * vs[page][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(seqs * heads, length, dim)
    # queries in a padded [sequence, row] grid
    row = torch.arange(most, device=q.device)[None]
    new = (cu[1:] - cu[:-1])[:, None]
    src = (cu[:-1, None] + row).clamp_max(q.shape[0] - 1)
    x = q[src].float().view(seqs, most, heads, group, dim).transpose(1, 2).reshape(seqs * heads, most * group, dim)
    s = torch.matmul(x, k).view(seqs, heads, most, group, length) * dim ** -0.5
    at = total[:, None] - new + row
    pos = torch.arange(length, device=q.device)
    seen = (pos <= at[..., None]) & (pos < total[:, None, None]) & ((pos > at[..., None] - case["window"]) | (pos < case["sinks"]))
    s = torch.where(seen[:, None, :, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = (s - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    out = torch.matmul(e.view(seqs * heads, most * group, length), v).view(seqs, heads, most, group, dim)
    out = out / e.sum(-1, keepdim=True).clamp_min(1e-30)
    out = out.transpose(1, 2).reshape(seqs, most, heads * group, dim)
    t = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return {"out": out[seq, t - cu[seq]].to(q.dtype)}


# ---- the definitions in 64 bits ----

def _exact_values(q, scale):
    sign = 1.0 - 2.0 * (q >> 3 & 1).double()
    e, f = (q >> 1 & 3).double(), (q & 1).double()
    mag = torch.where(e == 0, f / 2, torch.exp2(e - 1) * (1 + f / 2))
    s = torch.exp2(scale.double() - 127)
    s[scale == 255] = math.nan
    return sign * mag * s.repeat_interleave(32, -1)


def _exact_quantised(x):
    """The values that a row's codes and scales stand for."""
    x = x.double()
    out = torch.empty_like(x)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    for r in range(0, x.shape[0], 512):
        v = x[r:r + 512].reshape(-1, 32)
        top = v.abs().max(1).values
        scale = torch.exp2((torch.floor(torch.log2(top)) - 2).clamp(min=-127))
        u = (v.abs() / scale[:, None]).clamp(max=6)
        hi = torch.bucketize(u, levels).clamp(max=7)  # the first level at or above it
        lo = (hi - 1).clamp(min=0)
        down, up = u - levels[lo], levels[hi] - u
        code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
        y = levels[code] * torch.sign(v) * scale[:, None]
        y[~v.isfinite().all(1)] = math.nan
        out[r:r + 512] = y.view(-1, x.shape[1])
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quant":
        return {"values": _exact_quantised(state["x"])}
    if case["op"] in ("product", "linear"):
        def codes(q):
            return torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1)

        a = _exact_quantised(state["x"]) if case["op"] == "linear" else _exact_values(codes(state["a"]), state["scale_a"])
        parts, at = [], 0
        for rows in _pieces(case["n"]):
            w = _exact_values(codes(state["w"][at:at + rows]), state["scale_w"][at:at + rows])
            parts.append(a @ w.t().contiguous())
            at += rows
        return {"out": torch.cat(parts, 1)}

    lens = _lengths(case)
    if case["op"] == "rotate":
        r, out = case["rotary"], {}
        pos = torch.cat([torch.arange(s, s + n) for s, n in lens]).to(state["q"].device).double()
        # a pair as a complex number
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device=pos.device), pos[:, None] * state["freqs"][None])[:, None]
        for name, w in zip(("q", "k"), state["w"]):
            y = state[name].double()
            if w is not None:
                y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
            first = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
            second = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
        return out

    kc, vc, ks, vs = state["cache"]
    size, group, table = case["block"], case["heads"] // case["kv_heads"], state["table"].tolist()
    out, row = torch.empty(state["q"].shape, dtype=torch.float64, device=kc.device), 0
    for n_seq, (before, new) in enumerate(lens):
        n = before + new
        pages = torch.tensor(table[n_seq][:(n + size - 1) // size], device=kc.device)
        k = (_held(kc, pages).double() * ks[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
        v = (_held(vc, pages).double() * vs[pages].double()[..., None, None]).permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
        i = torch.arange(before, n, device=kc.device)[:, None]
        j = torch.arange(n, device=kc.device)[None]
        hidden = (j > i) | ((j <= i - case["window"]) & (j >= case["sinks"]))
        for h in range(case["heads"]):
            s = state["q"][row:row + new, h].double() @ k[h // group].t().contiguous() / math.sqrt(case["dim"])
            out[row:row + new, h] = torch.softmax(s.masked_fill_(hidden, -math.inf), -1) @ v[h // group].contiguous()
        row += new
    return {"out": out}
