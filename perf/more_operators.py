"""More operators around the attention kernels, measured one pass at a time.

    kv_cache_append                   q/k norm and rotation of new tokens, their keys and values into the paged cache, in one call
    kv_cache_write / kv_cache_read    over a cache held in 4 bits: e2m1 codes, an e4m3 scale every 16 values, an exponent byte a row
    fwd_decode                        over a cache held in 4 bits, and with first keys that stay visible beside a sliding window
    qk_norm_rope / qk_norm_rope_bwd   with positions of several axes (time, height, width), with the norm or without

`own = False` computes them in elementary torch operations, `own = True` through the package.  A case is a
dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` makes one pass, `exact` computes the
same outputs in 64 bits from the definitions.
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FP8 = torch.float8_e4m3fn
DEV = "cuda"
ROPE_BASE = 1e6
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------------------------------

def _rope(name, op, tokens, hq, hkv, d, rot, interleaved, axes, normed):
    return {"name": name, "op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "axes": axes, "normed": normed}


def _append(name, op, batch, max_len, hq, hkv, d, rot, interleaved, axes, normed, page, kv):
    return {"name": name, "op": op, "batch": batch, "max_len": max_len, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "axes": axes, "normed": normed, "page": page, "kv": kv}


def _cache(name, op, batch, max_len, hkv, d, page):
    return {"name": name, "op": op, "batch": batch, "max_len": max_len, "hkv": hkv, "d": d, "page": page, "kv": "e2m1"}


def _decode(name, batch, max_len, hq, hkv, d, page, kv, sink, first, window):
    return {"name": name, "op": "decode", "batch": batch, "max_len": max_len, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "kv": kv, "sink": sink, "first": first, "window": window}


def listed():
    return [
        # the new tokens of 48 requests of one decode step: a call whose latency counts
        _append("append, 48 new tokens, bf16", "append_step", 48, 8192, 64, 8, 128, 128, False, "", True, 64, "bf16"),
        # prompts of ragged lengths go into a 4-bit cache and come back as the next layer's attention reads them
        _append("append, prompts, 4 bits", "append", 8, 12000, 16, 4, 128, 128, False, "", True, 64, "e2m1"),
        # a short prompt of a model with head dim 64 into a 4-bit cache, and back
        _cache("cache in 4 bits, 1K, there and back", "write_read", 3, 500, 2, 64, 16),
        # the prompts of a batch into a 4-bit cache, and back
        _cache("cache in 4 bits, prompts, there and back", "write_read", 16, 16384, 8, 128, 64),
        # one interactive request at the start of its context
        _decode("decode in 4 bits, 1 x 777", 1, 777, 16, 4, 128, 16, "e2m1", False, 0, 0),
        # a full serving batch of ragged contexts
        _decode("decode in 4 bits, 64 x 16K", 64, 16384, 64, 8, 128, 64, "e2m1", False, 0, 0),
        # one request with a context of a million tokens
        _decode("decode in 4 bits, 1 x 1M", 1, 1048576, 16, 4, 128, 64, "e2m1", False, 0, 0),
        # a small batch of streaming requests: 4 first keys and the last thousand
        _decode("decode, 4 x 4K, first 4, window", 4, 4096, 64, 8, 128, 64, "e4m3", False, 4, 1024),
        # the sink + window mask of the 256K workload, one new token a document
        _decode("decode, 8 x 32K, first 1024, window", 8, 32768, 32, 32, 128, 64, "bf16", False, 1024, 4096),
        # the tokens of a few small images
        _rope("norm rope, 3 axes, 1K", "rope", 1001, 16, 4, 128, 128, False, "16,24,24", True),
        # the packed 128K video sequence, before its block-causal forward; the axes take turns over the pairs
        _rope("norm rope, 3 axes, 128K", "rope", 131072, 64, 8, 128, 128, False, "cyclic 3", True),
        # a quarter of it, after the attention's backward
        _rope("norm rope backward, 3 axes, 32K", "rope_bwd", 32768, 64, 8, 128, 128, False, "16,24,24", True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_axes(rng, rot):
    kind = rng.choice(["", "cyclic 3", "cyclic 2", "sections 3", "sections 3", "sections 4"])
    if not kind.startswith("sections"):
        return kind
    n, left, parts = int(kind[-1]), rot // 2, []
    for i in range(n - 1):
        parts.append(rng.randint(1, max(1, left - (n - 1 - i))))
        left -= parts[-1]
    return ",".join(str(x) for x in parts + [left])


def draw(rng: random.Random):
    op = rng.choice(["rope", "rope_bwd", "append", "append_step", "write_read", "decode", "decode", "decode4", "decode4"])
    d = rng.choice([64, 128])
    if op in ("rope", "rope_bwd"):
        hq, hkv = rng.choice([(16, 4), (32, 32), (64, 8), (6, 2), (3, 3), (5, 1)])
        tokens = _spread(rng, 1, 32768 * 72 * 128 // ((hq + hkv) * d))
        rot = rng.choice([d, d, d // 2, 16, 48])
        axes = _draw_axes(rng, rot)
        c = _rope("", op, tokens, hq, hkv, d, rot, rng.random() < 0.4, axes, axes != "" and rng.random() < 0.7)
    elif op in ("append", "append_step"):
        hq, hkv = rng.choice([(16, 4), (32, 32), (64, 8), (6, 2), (3, 3), (5, 1)])
        batch = _spread(rng, 1, 128)
        most = max(1, 8 * 12000 * 20 * 128 // (batch * (hq + hkv) * d))
        rot = rng.choice([d, d, d // 2, 16, 48])
        c = _append("", op, batch, _spread(rng, 1, min(most, 65536)), hq, hkv, d, rot, rng.random() < 0.4,
                    rng.choice(["", _draw_axes(rng, rot)]), rng.random() < 0.7, rng.choice([16, 32, 64, 128]),
                    rng.choice(["bf16", "e4m3", "e2m1"]))
    elif op == "write_read":
        hkv = rng.choice([1, 2, 3, 4, 8, 32])
        batch = _spread(rng, 1, 128)
        most = max(1, 16 * 16384 * 8 * 64 // (batch * hkv * d))
        c = _cache("", op, batch, _spread(rng, 1, min(most, 65536)), hkv, d, rng.choice([16, 32, 64, 128]))
    else:
        hq, hkv = rng.choice([(16, 4), (16, 4), (64, 8), (32, 32), (8, 1), (6, 2), (3, 3), (32, 2)])
        batch = _spread(rng, 1, 256)
        most = max(16, min(1 << 20, 64 * 16384 * 8 * 64 // (batch * hkv * d)))
        max_len = _spread(rng, 1, most)
        first, window = (rng.choice([1, 4, 37, 500]), max(1, max_len // 3)) if op == "decode" or rng.random() < 0.3 else (0, 0)
        c = _decode("", batch, max_len, hq, hkv, d, rng.choice([16, 32, 64, 128]),
                    rng.choice(["bf16", "e4m3"]) if op == "decode" else "e2m1", rng.random() < 0.3, first, window)
    del c["name"]
    return c


def _lens(case):
    """Lengths of the batch's sequences, by the case alone: ragged, the longest first."""
    b, top = case["batch"], case["max_len"]
    if b == 1:
        return np.array([top], dtype=np.int64)
    r = np.random.RandomState((1009 * b + top) % (1 << 31))
    lens = np.maximum(1, (top * r.uniform(0.25, 1.0, b)).astype(np.int64))
    lens[0] = top
    return lens


def _pair_axes(case):
    """The axis of each rotation pair, a list of rot / 2 numbers."""
    n, text = case["rot"] // 2, case["axes"]
    if not text:
        return [0] * n
    if text.startswith("cyclic"):
        return [i % int(text.split()[1]) for i in range(n)]
    return [a for a, c in enumerate(text.split(",")) for _ in range(int(c))]


def _stored_bytes(case):
    d = case["d"]
    return {"bf16": 2 * d, "e4m3": d + 1, "e2m1": d // 2 + d // 16 + 1}[case["kv"]]


def _visible(case):
    """Keys that a new token sees, summed over the batch."""
    lens = _lens(case)
    if not case["window"]:
        return int(lens.sum())
    starts = np.maximum(lens - case["window"], 0)
    return int((np.minimum(case["first"], starts) + lens - starts).sum())


def work(case):
    op, d = case["op"], case["d"]
    n_axes = max(_pair_axes(case)) + 1 if "axes" in case else 1
    if op in ("rope", "rope_bwd"):
        rows, weights = case["tokens"] * (case["hq"] + case["hkv"]), 8 * d if case["normed"] else 0
        each = 4 if op == "rope" or not case["normed"] else 6
        # of the table each token's rows are counted, up to a table of so many rows as there are tokens
        table = 4 * case["rot"] * min(case["tokens"], _max_pos(case)) + 4 * n_axes * case["tokens"]
        return {"bytes": rows * d * each + table + weights * (1 if op == "rope" else 2),
                "flops": rows * ((4 if op == "rope" else 11) * d * case["normed"] + 3 * case["rot"])}
    lens = _lens(case)
    total = int(lens.sum())
    if op in ("append", "append_step"):
        tokens = case["batch"] if op == "append_step" else total
        kv_rows = 2 * case["hkv"] * tokens
        table = 4 * case["rot"] * min(tokens, _max_pos(case)) + 4 * n_axes * tokens + 8 * tokens
        nbytes = tokens * case["hq"] * 4 * d + kv_rows * (2 * d + _stored_bytes(case)) + table + 8 * d * case["normed"]
        if case["kv"] != "bf16":
            nbytes += kv_rows * (2 * d + _stored_bytes(case))
        return {"bytes": nbytes, "flops": tokens * (case["hq"] + case["hkv"]) * (4 * d * case["normed"] + 3 * case["rot"])}
    if op == "write_read":
        rows = 2 * case["hkv"] * total
        return {"bytes": 2 * rows * (2 * d + _stored_bytes(case)) + 12 * total, "flops": rows * d * 4}
    keys = _visible(case)
    return {"bytes": 2 * keys * case["hkv"] * _stored_bytes(case) + case["batch"] * case["hq"] * (4 * d + 4),
            "flops": 4 * keys * case["hq"] * d}


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _table(max_pos, rot):
    """cos and sin of pos * base^(-2i / rot), angles in 64 bits: [max_pos, rot] with the cosines first."""
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, device=DEV, dtype=F64) / rot)
    ang = torch.arange(max_pos, device=DEV, dtype=F64)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _max_pos(case):
    if case["op"] in ("rope", "rope_bwd"):
        return 32768
    return case["max_len"] + 64


def _positions(case, seq_pos, g):
    """int32 [tokens], or [axes, tokens]: frames of 48 x 80 patches behind each other, or a place of its own for a lone token."""
    axes = max(_pair_axes(case)) + 1
    if not case["axes"]:
        return seq_pos.to(torch.int32)
    top = _max_pos(case)
    rows = [seq_pos // 3840, seq_pos // 80 % 48, seq_pos % 80, seq_pos % 7]
    shift = torch.randint(0, 64, (axes, 1), generator=g, device=DEV)
    return (torch.stack(rows[:axes]) + shift).clamp(max=top - 1).to(torch.int32)


def _pages(lens, page, g):
    """A page table of pages in random order, -1 behind each sequence's last page, and the number of pages."""
    need = (lens + page - 1) // page
    total, width = int(need.sum()), max(1, int(need.max()))
    order = torch.randperm(total + 3, generator=g, device=DEV).to(torch.int32)[:total]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    has = torch.arange(width, device=DEV)[None, :] < torch.from_numpy(need).to(DEV)[:, None]
    table[has] = order
    return table, total + 3


def _empty_cache(shape, kv):
    """(rows, scales, exponent bytes) of a cache [pages, heads, page, d], all zeros."""
    d = shape[3]
    if kv == "bf16":
        return torch.zeros(shape, dtype=BF16, device=DEV), None, None
    exps = torch.zeros(shape[:3], dtype=torch.uint8, device=DEV)
    if kv == "e4m3":
        return torch.zeros(shape, dtype=FP8, device=DEV), None, exps
    return (torch.zeros(shape[:3] + (d // 2,), dtype=torch.uint8, device=DEV),
            torch.zeros(shape[:3] + (d // 16,), dtype=FP8, device=DEV), exps)


def _random_cache(shape, g, spread, kv):
    """A cache [pages, heads, page, d] that has been written before."""
    rows, scales, exps = _empty_cache(shape, kv)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):
        some = (min(step, shape[0] - i),) + shape[1:]
        x = torch.randn(some, generator=g, device=DEV, dtype=BF16)
        x *= torch.exp(spread * torch.randn(some[:3] + (1,), generator=g, device=DEV)).to(BF16)
        parts = _store(x, kv)
        for into, part in zip((rows, scales, exps), parts):
            if into is not None:
                into[i:i + step] = part
    return rows, scales, exps


def prepare(case, seed):
    g = _generator(seed)
    op, d = case["op"], case["d"]
    s = {"case": case}
    if op in ("rope", "rope_bwd", "append", "append_step"):
        if op in ("rope", "rope_bwd"):
            t = case["tokens"]
            at = torch.arange(t, device=DEV) if t >= 1024 or case["axes"] else torch.randint(0, _max_pos(case), (t,), generator=g, device=DEV)
            s["positions"] = _positions(case, at % _max_pos(case), g)
        else:
            lens = _lens(case)
            s["page_table"], pages = _pages(lens, case["page"], g)
            lens_d = torch.from_numpy(lens).to(DEV)
            if op == "append_step":
                seq, pos = torch.arange(len(lens), device=DEV), lens_d - 1
            else:
                seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lens_d)
                pos = torch.arange(int(lens.sum()), device=DEV) - (lens_d.cumsum(0) - lens_d)[seq]
                s["cu_seqlens"] = torch.cat([lens_d.new_zeros(1), lens_d.cumsum(0)]).to(torch.int32)
            t, page = len(seq), case["page"]
            s["slots"] = s["page_table"][seq, pos // page].long() * page + pos % page
            s["positions"] = _positions(case, pos, g)
            if op == "append_step" and case["kv"] != "bf16":   # what comes back is the page rows' first keys, one a sequence
                s["page_table"] = (s["slots"] // page).to(torch.int32)[:, None]
                s["cu_seqlens"] = torch.cat([lens_d.new_zeros(1), (pos % page + 1).cumsum(0)]).to(torch.int32)
            s["total"] = int(s["cu_seqlens"][-1]) if "cu_seqlens" in s else 0
            shape = (pages, case["hkv"], page, d)
            for n in "kv":
                s[n + "_cache"], s[n + "_scale"], s[n + "_exp"] = _empty_cache(shape, case["kv"])
        hq, hkv = case["hq"], case["hkv"]
        # one fused projection's output: q, k and v are views of it, a few columns larger than the rest
        qkv = torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEV, dtype=BF16)
        qkv *= (1.0 + 4.0 * (torch.rand(d, generator=g, device=DEV) < 0.03)).to(BF16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * torch.randn(2, d, generator=g, device=DEV)).unbind(0) if case["normed"] else (None, None)
        s["table"] = _table(_max_pos(case), case["rot"])
        s["axes"] = _pair_axes(case) if case["axes"] else None
        if op == "rope_bwd":
            s["dq_out"] = 0.1 * torch.randn(t, hq, d, generator=g, device=DEV, dtype=BF16)
            s["dk_out"] = 0.1 * torch.randn(t, hkv, d, generator=g, device=DEV, dtype=BF16)
        return s
    lens = _lens(case)
    page, hkv = case["page"], case["hkv"]
    s["page_table"], pages = _pages(lens, page, g)
    shape = (pages, hkv, page, d)
    lens_d = torch.from_numpy(lens).to(DEV)
    if op == "write_read":
        for n in "kv":
            s[n + "_cache"], s[n + "_scale"], s[n + "_exp"] = _empty_cache(shape, case["kv"])
        seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lens_d)
        pos = torch.arange(int(lens.sum()), device=DEV) - (lens_d.cumsum(0) - lens_d)[seq]
        s["slots"] = s["page_table"][seq, pos // page].long() * page + pos % page
        s["cu_seqlens"] = torch.cat([lens_d.new_zeros(1), lens_d.cumsum(0)]).to(torch.int32)
        s["total"] = int(lens.sum())
        s["k"] = torch.randn(s["total"], hkv, d, generator=g, device=DEV, dtype=BF16)
        kv = torch.randn(s["total"], 2 * hkv, d, generator=g, device=DEV, dtype=BF16)   # v stays in the projection's output
        kv *= torch.exp(torch.randn(s["total"], 2 * hkv, 1, generator=g, device=DEV)).to(BF16)
        s["v"] = kv[:, hkv:]
        return s
    s["k_cache"], s["k_scale"], s["k_exp"] = _random_cache(shape, g, 0.1, case["kv"])
    s["v_cache"], s["v_scale"], s["v_exp"] = _random_cache(shape, g, 0.7, case["kv"])
    s["q"] = torch.randn(case["batch"], case["hq"], d, generator=g, device=DEV, dtype=BF16)
    s["kv_lens"] = lens_d.to(torch.int32)
    s["kv_starts"] = (lens_d - case["window"]).clamp(min=0).to(torch.int32) if case["window"] else None
    s["kv_firsts"] = torch.full_like(s["kv_lens"], case["first"]) if case["window"] else None
    s["sink"] = torch.randn(case["hq"], generator=g, device=DEV) if case["sink"] else None
    s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import flexible_mask_flashattention_gb300 as ffa
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return ffa.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"], eps=EPS,
                                interleaved=case["interleaved"], axes=s["axes"])
    if op == "rope_bwd":
        grads = ffa.qk_norm_rope_bwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"],
                                     s["dq_out"], s["dk_out"], eps=EPS, interleaved=case["interleaved"], axes=s["axes"])
        return grads if case["normed"] else grads[:2]
    more = {n: s[n] for n in ("k_exp", "v_exp", "k_scale", "v_scale")}
    if op in ("append", "append_step"):
        q = ffa.kv_cache_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["table"], s["positions"],
                                s["k_cache"], s["v_cache"], s["slots"], eps=EPS, interleaved=case["interleaved"],
                                axes=s["axes"], **more)
        if case["kv"] == "bf16":
            return q, s["k_cache"], s["v_cache"]
    if op == "write_read":
        ffa.kv_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], **more)
    if op != "decode":
        k, v = ffa.kv_cache_read(s["k_cache"], s["v_cache"], s["page_table"], s["cu_seqlens"], s["total"], **more)
        return (k, v) if op == "write_read" else (q, k, v)
    return ffa.fwd_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["scale"],
                          kv_starts=s["kv_starts"], kv_firsts=s["kv_firsts"], sink=s["sink"], **more)


def _pairs(x, rot, interleaved):
    """The two halves of the rotated columns' pairs, and the columns behind them."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    return a, b, x[..., rot:]


def _unpairs(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _cos_sin(s):
    half = s["case"]["rot"] // 2
    if s["axes"] is None:
        cs = s["table"][s["positions"].long()][:, None, :]
        return cs[..., :half], cs[..., half:]
    at = s["positions"][torch.tensor(s["axes"], device=DEV)].t().long()   # [tokens, pairs]
    pair = torch.arange(half, device=DEV)
    return s["table"][at, pair][:, None, :], s["table"][at, half + pair][:, None, :]


def _norm_rope(s, x, w):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    cos, sin = _cos_sin(s)
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    a, b, rest = _pairs(y, rot, inter)
    return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, inter).to(BF16)


def _norm_rope_bwd(s, x, w, dout):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    cos, sin = _cos_sin(s)
    a, b, rest = _pairs(dout.float(), rot, inter)
    dy = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, inter)
    if w is None:
        return dy.to(BF16), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dw = (dy * xh).sum((0, 1))
    dy = dy * w
    return (r * (dy - xh * (dy * xh).mean(-1, keepdim=True))).to(BF16), dw


def _pow2(n):
    """2^n in 32 bits, exactly, for -126 <= n <= 127."""
    return ((n.int() + 127) << 23).view(F32)


def _least_exponent(x, most_fraction, most_exponent):
    """The smallest n >= -126 with max|x| <= most_fraction * 2^most_exponent * 2^n, a row; most_fraction in [0.5, 1)."""
    f, e = torch.frexp(x.abs().amax(-1))
    return torch.where(f <= most_fraction, e - most_exponent, e - most_exponent + 1).clamp(min=-126)


def _e2m1_codes(z):
    """The nearest e2m1 code of each z, ties to the even code: values 0, 0.5, 1, 1.5, 2, 3, 4, 6, and the sign bit 8."""
    a = z.abs().clamp(max=6.0)
    code = torch.where(a < 2.0, torch.round(2.0 * a), torch.where(a < 4.0, 2.0 + torch.round(a), 4.0 + torch.round(0.5 * a)))
    return code.to(torch.uint8) + 8 * torch.signbit(z).to(torch.uint8)


def _store(x, kv):
    """Rows as a cache stores them: (rows or codes, scales or None, exponent bytes or None)."""
    if kv == "bf16":
        return x, None, None
    x = x.float()
    if kv == "e4m3":   # 448 = 0.875 * 2^9
        n = _least_exponent(x, 0.875, 9)
        return (x * _pow2(-n)[..., None]).to(FP8), None, (n + 127).to(torch.uint8)
    n = _least_exponent(x, 0.65625, 12)   # 6 * 448 = 0.65625 * 2^12
    y = (x * _pow2(-n)[..., None]).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6.0).to(FP8)
    z = torch.where(scale.float()[..., None] > 0.0, y / scale.float()[..., None], torch.copysign(torch.zeros_like(y), y))
    codes = _e2m1_codes(z).flatten(-2)
    return codes[..., 0::2] + 16 * codes[..., 1::2], scale, (n + 127).to(torch.uint8)


def _stored(rows, scales, exps):
    """What stored rows stand for, in 32 bits."""
    if exps is None:
        return rows.float()
    if scales is None:
        return rows.float() * _pow2(exps.int() - 127)[..., None]
    code = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).int()
    low, high = code & 1, (code >> 1) & 3
    v = torch.where(high == 0, 0.5 * low, (1.0 + 0.5 * low) * 0.5 * (1 << high)) * (1.0 - 2.0 * (code >> 3))
    return (v.unflatten(-1, (-1, 16)) * scales.float()[..., None]).flatten(-2) * _pow2(exps.int() - 127)[..., None]


def _put(cache, at, off, x):
    """cache[page, :, offset] = rows, of any type."""
    if cache is not None:
        (cache.view(torch.uint8) if cache.dtype == FP8 else cache)[at, :, off] = x.view(torch.uint8) if cache.dtype == FP8 else x


def _take(cache, *at):
    if cache is None:
        return None
    return cache.view(torch.uint8)[at].view(FP8) if cache.dtype == FP8 else cache[at]


def _write_plain(s, k, v):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    for n, x in (("k", k), ("v", v)):
        rows, scales, exps = _store(x, s["case"]["kv"])
        _put(s[n + "_cache"], at, off, rows)
        _put(s[n + "_scale"], at, off, scales)
        _put(s[n + "_exp"], at, off, exps)


def _read_plain(s):
    page, cu = s["case"]["page"], s["cu_seqlens"].long()
    row = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = row - cu[seq]
    where = (s["page_table"][seq, pos // page].long(), slice(None), pos % page)
    return tuple(_stored(*(_take(s[n + part], *where) for part in ("_cache", "_scale", "_exp"))).to(BF16) for n in "kv")


def _run_plain(s):
    op = s["case"]["op"]
    if op == "rope":
        return _norm_rope(s, s["q"], s["q_weight"]), _norm_rope(s, s["k"], s["k_weight"])
    if op == "rope_bwd":
        dq, dqw = _norm_rope_bwd(s, s["q"], s["q_weight"], s["dq_out"])
        dk, dkw = _norm_rope_bwd(s, s["k"], s["k_weight"], s["dk_out"])
        return (dq, dk) if dqw is None else (dq, dk, dqw, dkw)
    if op in ("append", "append_step"):
        q = _norm_rope(s, s["q"], s["q_weight"])
        _write_plain(s, _norm_rope(s, s["k"], s["k_weight"]), s["v"])
        return (q, s["k_cache"], s["v_cache"]) if s["case"]["kv"] == "bf16" else (q, *_read_plain(s))
    if op == "write_read":
        _write_plain(s, s["k"], s["v"])
        return _read_plain(s)
    return _decode_plain(s)


def _decode_plain(s):
    q = s["q"].float()
    b, hq, d = q.shape
    table = s["page_table"].clamp(min=0).long()
    hkv = s["case"]["hkv"]

    def padded(n):   # [b, hkv, keys, d] of every sequence's pages
        x = _stored(*(_take(s[n + part], table) for part in ("_cache", "_scale", "_exp")))
        return x.transpose(1, 2).reshape(b, hkv, -1, d)

    k = padded("k")
    logits = torch.matmul(q.view(b, hkv, -1, d), k.transpose(-1, -2)).mul_(s["scale"])
    del k
    j = torch.arange(logits.shape[-1], device=DEV)
    keep = j[None, :] < s["kv_lens"][:, None]
    if s["kv_starts"] is not None:
        keep &= (j[None, :] >= s["kv_starts"][:, None]) | (j[None, :] < s["kv_firsts"][:, None])
    keep = keep[:, None, None, :]
    logits = torch.where(keep, logits, -math.inf)
    m = logits.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, hkv, -1, 1)
        m = torch.maximum(m, sink)
    p = torch.where(keep, torch.exp(logits - m), 0.0)
    total = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - m)
    v = torch.where(keep.transpose(-1, -2), padded("v"), 0.0)
    out = torch.matmul(p, v) / total
    lse = (m + torch.log(total)).view(b, hq).t().contiguous()
    return out.view(b, hq, d).to(BF16), lse


# ---- the same in 64 bits, from the definitions ----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("rope", "rope_bwd"):
            return _exact_rope(s)
        if op in ("append", "append_step"):
            return _exact_append(s)
        return _exact_write_read(s) if op == "write_read" else _exact_decode(s)


def _exact_matrix(s, rows):
    """The rotation of each of `rows` as a dense matrix [n, d, d] in 64 bits."""
    d, rot = s["case"]["d"], s["case"]["rot"]
    i = torch.arange(rot // 2, device=DEV)
    a, b = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + rot // 2)
    pos = s["positions"] if s["positions"].dim() == 2 else s["positions"][None]
    n = len(range(*rows.indices(pos.shape[1])))
    m = torch.eye(d, dtype=F64, device=DEV).repeat(n, 1, 1)
    for axis, p in enumerate(pos):
        mine = torch.tensor([k for k, x in enumerate(_pair_axes(s["case"])) if x == axis], dtype=torch.int64, device=DEV)
        cs = s["table"].to(F64)[p[rows].long()]
        c, sn, x, y = cs[:, mine], cs[:, rot // 2 + mine], a[mine], b[mine]
        m[:, x, x], m[:, y, y], m[:, x, y], m[:, y, x] = c, c, -sn, sn
    return m


def _exact_rope_of(s, name):
    """out = M diag(w) x / |x|rms, with M the position's rotation matrix; gradients by the chain rule through M, w and the norm."""
    x_all, w = s[name], s[name + "_weight"]
    d, back = s["case"]["d"], s["case"]["op"] == "rope_bwd"
    parts, dw = [], torch.zeros(d, dtype=F64, device=DEV)
    for i in range(0, x_all.shape[0], 4096):
        rows = slice(i, min(x_all.shape[0], i + 4096))
        m = _exact_matrix(s, rows)
        x = x_all[rows].to(F64)
        rms = (torch.einsum("thd,thd->th", x, x) / d + EPS).sqrt()[..., None]
        if not back:
            parts.append(torch.bmm(x if w is None else w.to(F64) * (x / rms), m.transpose(1, 2)))
            continue
        g = torch.bmm(s["d" + name + "_out"][rows].to(F64), m)
        if w is not None:
            dw += torch.einsum("thd,thd->d", g, x / rms)
            g = g * w.to(F64)
            g = g / rms - x * torch.einsum("thd,thd->th", g, x)[..., None] / (d * rms ** 3)
        parts.append(g)
    return torch.cat(parts), dw


def _exact_rope(s):
    (q, dqw), (k, dkw) = _exact_rope_of(s, "q"), _exact_rope_of(s, "k")
    return (q, k, dqw, dkw) if s["case"]["op"] == "rope_bwd" and s["case"]["normed"] else (q, k)


E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_VALUES = tuple(sorted({(m / 8.0 + (1 if e else 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)
                            if (e, m) != (15, 7)}))


def _power(n):
    """2^n in 64 bits, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(F64)


def _nearest(x, values):
    """The nearest of the values, ties to the even place in their order; beyond the last: the last."""
    grid = torch.tensor(values, dtype=F64, device=DEV)
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.sign(x) * torch.where(up, grid[hi], grid[lo])


def _exact_stored(x, kv):
    """What rows of 16-bit values become by being stored, in 64 bits."""
    if kv == "bf16":
        return x
    most = 448.0 if kv == "e4m3" else 2688.0
    top = x.abs().max(-1).values
    e = torch.full_like(top, -126.0)
    some = top > 0
    e[some] = torch.ceil(torch.log2(top[some] / most))
    e = torch.where(top <= most * _power(e - 1), e - 1, torch.where(top > most * _power(e), e + 1, e)).clamp(min=-126)
    y = x / _power(e)[..., None]
    if kv == "e4m3":
        y = _nearest(y, E4M3_VALUES)
    else:
        y = y.unflatten(-1, (-1, 16))
        scale = _nearest(y.abs().max(-1).values / 6.0, E4M3_VALUES)[..., None]
        y = (_nearest(torch.where(scale > 0, y / scale.clamp(min=1e-30), torch.zeros_like(y)), E2M1_VALUES) * scale).flatten(-2)
    return y * _power(e)[..., None]


def _exact_kept(s, k, v, read):
    """The cache after k and v are written to it: whole, or as reading it back gives it (rows that no token wrote are 0)."""
    case, page = s["case"], s["case"]["page"]
    outs = []
    for x, n in ((k, "k"), (v, "v")):
        cache = torch.zeros(s[n + "_exp"].shape + (case["d"],) if s[n + "_exp"] is not None else s[n + "_cache"].shape, dtype=F64, device=DEV)
        for i in range(0, len(s["slots"]), 16384):
            slots = s["slots"][i:i + 16384]
            cache[slots // page, :, slots % page] = _exact_stored(x[i:i + 16384].to(F64), case["kv"])
        if read:
            cu, rows = s["cu_seqlens"].tolist(), []
            for b in range(len(cu) - 1):
                pages = s["page_table"][b, :(cu[b + 1] - cu[b] + page - 1) // page].long()
                rows.append(cache[pages].transpose(1, 2).flatten(0, 1)[:cu[b + 1] - cu[b]])
            cache = torch.cat(rows)
        outs.append(cache)
    return tuple(outs)


def _exact_append(s):
    q, _ = _exact_rope_of(s, "q")
    k, _ = _exact_rope_of(s, "k")
    # a key is a 16-bit value before it is stored in fewer
    k = k if s["case"]["kv"] == "bf16" else k.to(BF16).to(F64)
    return (q, *_exact_kept(s, k, s["v"].to(F64), s["case"]["kv"] != "bf16"))


def _exact_write_read(s):
    return _exact_kept(s, s["k"], s["v"], True)


def _exact_rows(s, n, b, at):
    """Rows `at` (positions) of sequence b in 64 bits: [keys, hkv, d]."""
    page, kv = s["case"]["page"], s["case"]["kv"]
    where = (s["page_table"][b, at // page].long(), slice(None), at % page)
    x = _take(s[n + "_cache"], *where)
    if kv == "bf16":
        return x.to(F64)
    if kv == "e2m1":
        values = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), dtype=F64, device=DEV)
        x = torch.stack([values[(x % 16).long()], values[torch.div(x, 16, rounding_mode="floor").long()]], -1).flatten(-2)
        x = x * torch.repeat_interleave(_take(s[n + "_scale"], *where).to(F64), 16, -1)
    return x.to(F64) * _power(s[n + "_exp"][where].to(torch.int64) - 127)[..., None]


def _exact_decode(s):
    case = s["case"]
    lens, hkv, d = s["kv_lens"].tolist(), case["hkv"], case["d"]
    starts = s["kv_starts"].tolist() if s["kv_starts"] is not None else [0] * len(lens)
    outs, lses = [], []
    for b, (lo, hi) in enumerate(zip(starts, lens)):
        at = torch.cat([torch.arange(min(case["first"], lo), device=DEV), torch.arange(lo, hi, device=DEV)])
        q = s["q"][b].to(F64).view(hkv, -1, d)
        z = torch.einsum("hgd,khd->hgk", q, _exact_rows(s, "k", b, at)) * s["scale"]
        if s["sink"] is not None:
            z = torch.cat([z, s["sink"].to(F64).view(hkv, -1, 1)], -1)
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - lse[..., None])[..., :len(at)]
        outs.append(torch.einsum("hgk,khd->hgd", p, _exact_rows(s, "v", b, at)).reshape(-1, d))
        lses.append(lse.reshape(-1))
    return torch.stack(outs), torch.stack(lses, 1)
