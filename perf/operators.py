"""Operators around the attention kernels, measured one pass at a time.

    qk_norm_rope / qk_norm_rope_bwd   RMS norm of every q and k head row, with the position rotation in the same pass
    kv_cache_write / kv_cache_read    rows into a paged key-value cache (bf16, or e4m3 with a power-of-two scale a row), and back
    fwd_decode                        attention of one new token a sequence over the paged cache

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


# ---- cases ----------------------------------------------------------------------------------------------------------

def _norm(name, op, tokens, hq, hkv, d, rot, interleaved, max_pos):
    return {"name": name, "op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "max_pos": max_pos}


def _cache(name, op, batch, max_len, hkv, d, page, fp8):
    return {"name": name, "op": op, "batch": batch, "max_len": max_len, "hkv": hkv, "d": d, "page": page, "fp8": fp8}


def _decode(name, batch, max_len, hq, hkv, d, page, fp8, sink, window):
    return {"name": name, "op": "decode", "batch": batch, "max_len": max_len, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "fp8": fp8, "sink": sink, "window": window}


def listed():
    return [
        # the new token of each of 16 requests, before its attention step: a call whose latency counts
        _norm("norm rope, 16 new tokens", "norm", 16, 16, 4, 128, 128, False, 131072),
        # the packed 64K sequence of the varlen workload, before the forward
        _norm("norm rope, 64K tokens", "norm", 65536, 16, 4, 128, 128, False, 16384),
        # a small training batch of a model with head dim 64, pairs side by side and half of each head rotated
        _norm("norm rope backward, 2K", "norm_bwd", 2049, 6, 2, 64, 32, True, 2049),
        # the 64K sequence again, after the attention's backward
        _norm("norm rope backward, 64K", "norm_bwd", 65536, 16, 4, 128, 128, False, 16384),
        # one decode step of 48 requests: one row a request goes into its page
        _cache("cache write, 48 new tokens", "write_step", 48, 8192, 8, 128, 64, True),
        # prompts of ragged lengths go into their pages, quantised
        _cache("cache write, prompts, e4m3", "write", 16, 16384, 8, 128, 64, True),
        # a short prefix of a model with head dim 64 is read back for the next chunk's prefill
        _cache("cache read, 1K, bf16", "read", 3, 500, 2, 64, 16, False),
        # the prefixes of a batch are read back from a quantised cache
        _cache("cache read, prefixes, e4m3", "read", 16, 16384, 8, 128, 64, True),
        # one interactive request at the start of its context
        _decode("decode, 1 x 777, bf16", 1, 777, 16, 4, 128, 16, False, False, 0),
        # a serving batch with head dim 64, every head with keys of its own, sink logits and a sliding window
        _decode("decode, 24 x 8K, sink, window", 24, 8192, 32, 32, 64, 32, False, True, 4096),
        # a full serving batch of ragged contexts over a quantised cache
        _decode("decode, 64 x 16K, e4m3", 64, 16384, 64, 8, 128, 64, True, False, 0),
        # one request with a context of a million tokens
        _decode("decode, 1 x 1M, e4m3", 1, 1048576, 16, 4, 128, 64, True, False, 0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "norm_bwd", "write", "write_step", "read", "decode", "decode"])
    d = rng.choice([64, 128])
    if op in ("norm", "norm_bwd"):
        hq, hkv = rng.choice([(16, 4), (32, 32), (64, 8), (6, 2), (3, 3), (5, 1)])
        most = 65536 * 20 * 128 // ((hq + hkv) * d)
        tokens = _spread(rng, 1, most)
        rot = rng.choice([d, d, d // 2, 16, 48])
        c = _norm("", op, tokens, hq, hkv, d, rot, rng.random() < 0.4, _spread(rng, max(2, tokens // 8), 131072 + tokens))
    elif op in ("write", "write_step", "read"):
        hkv = rng.choice([1, 2, 3, 4, 8, 32])
        batch = _spread(rng, 1, 128)
        most = max(1, 16 * 16384 * 8 * 64 // (batch * hkv * d))
        c = _cache("", op, batch, _spread(rng, 1, min(most, 65536)), hkv, d, rng.choice([16, 32, 64, 128]), rng.random() < 0.6)
    else:
        hq, hkv = rng.choice([(16, 4), (16, 4), (64, 8), (32, 32), (8, 1), (6, 2), (3, 3), (32, 2)])
        batch = _spread(rng, 1, 256)
        most = max(16, min(1 << 20, 64 * 16384 * 8 * 64 // (batch * hkv * d)))
        max_len = _spread(rng, 1, most)
        window = rng.choice([0, 0, max(1, max_len // 3)])
        c = _decode("", batch, max_len, hq, hkv, d, rng.choice([16, 32, 64, 128]), rng.random() < 0.6,
                    rng.random() < 0.3, window)
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


def _row_bytes(case):
    return case["d"] * (1 if case["fp8"] else 2) + (1 if case["fp8"] else 0)


def work(case):
    op, d = case["op"], case["d"]
    if op in ("norm", "norm_bwd"):
        rows = case["tokens"] * (case["hq"] + case["hkv"])
        table = 4 * case["rot"] * min(case["tokens"], case["max_pos"]) + 4 * case["tokens"]
        if op == "norm":
            return {"bytes": rows * d * 4 + table + 8 * d, "flops": rows * (4 * d + 3 * case["rot"])}
        return {"bytes": rows * d * 6 + table + 16 * d, "flops": rows * (11 * d + 3 * case["rot"])}
    lens = _lens(case)
    if op in ("write", "write_step", "read"):
        rows = 2 * case["hkv"] * (case["batch"] if op == "write_step" else int(lens.sum()))
        ids = 8 * rows // (2 * case["hkv"]) if op != "read" else 4 * int(((lens + case["page"] - 1) // case["page"]).sum())
        return {"bytes": rows * (2 * d + _row_bytes(case)) + ids, "flops": rows * d * 2}
    keys = int((np.minimum(lens, case["window"]) if case["window"] else lens).sum())
    return {"bytes": 2 * keys * case["hkv"] * _row_bytes(case) + case["batch"] * case["hq"] * (4 * d + 4),
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


def _pages(lens, page, g):
    """A page table of pages in random order, -1 behind each sequence's last page, and the number of pages."""
    need = (lens + page - 1) // page
    total, width = int(need.sum()), max(1, int(need.max()))
    order = torch.randperm(total + 3, generator=g, device=DEV).to(torch.int32)[:total]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    has = torch.arange(width, device=DEV)[None, :] < torch.from_numpy(need).to(DEV)[:, None]
    table[has] = order
    return table, total + 3


def _random_cache(shape, g, spread, fp8):
    """A cache [pages, heads, page, d] that has been written before, in its stored form: (values, exponent bytes or None)."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=BF16)
    x *= torch.exp(spread * torch.randn(shape[:3] + (1,), generator=g, device=DEV)).to(BF16)
    if not fp8:
        return x, None
    codes = torch.empty(shape, dtype=FP8, device=DEV)
    exps = torch.empty(shape[:3], dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):
        codes[i:i + step], exps[i:i + step] = _quantise(x[i:i + step])
    return codes, exps


def prepare(case, seed):
    g = _generator(seed)
    op, d = case["op"], case["d"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        # one fused projection's output: q and k are views of it, a few columns larger than the rest
        qkv = torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEV, dtype=BF16)
        qkv *= (1.0 + 4.0 * (torch.rand(d, generator=g, device=DEV) < 0.03)).to(BF16)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["q_weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["k_weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["table"] = _table(case["max_pos"], case["rot"])
        if t < 1024:   # new tokens, each somewhere in its own context
            s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV, dtype=torch.int32)
        else:          # packed sequences, each counted from its start
            s["positions"] = (torch.arange(t, device=DEV) % case["max_pos"]).to(torch.int32)
        if op == "norm_bwd":
            s["dq_out"] = 0.1 * torch.randn(t, hq, d, generator=g, device=DEV, dtype=BF16)
            s["dk_out"] = 0.1 * torch.randn(t, hkv, d, generator=g, device=DEV, dtype=BF16)
        return s
    lens = _lens(case)
    page, hkv, fp8 = case["page"], case["hkv"], case["fp8"]
    s["page_table"], pages = _pages(lens, page, g)
    shape = (pages, hkv, page, d)
    lens_d = torch.from_numpy(lens).to(DEV)
    if op in ("write", "write_step"):
        s["k_cache"] = torch.zeros(shape, dtype=FP8 if fp8 else BF16, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["k_exp"], s["v_exp"] = (torch.zeros(shape[:3], dtype=torch.uint8, device=DEV) if fp8 else None for _ in "kv")
        if op == "write_step":
            seq, pos = torch.arange(len(lens), device=DEV), lens_d - 1
        else:
            seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lens_d)
            pos = torch.arange(int(lens.sum()), device=DEV) - (lens_d.cumsum(0) - lens_d)[seq]
        s["slots"] = s["page_table"][seq, pos // page].long() * page + pos % page
        t = len(seq)
        s["k"] = torch.randn(t, hkv, d, generator=g, device=DEV, dtype=BF16)
        kv = torch.randn(t, 2 * hkv, d, generator=g, device=DEV, dtype=BF16)   # v stays in the projection's output
        kv *= torch.exp(torch.randn(t, 2 * hkv, 1, generator=g, device=DEV)).to(BF16)
        s["v"] = kv[:, hkv:]
        return s
    s["k_cache"], s["k_exp"] = _random_cache(shape, g, 0.1, fp8)
    s["v_cache"], s["v_exp"] = _random_cache(shape, g, 0.7, fp8)
    if op == "read":
        s["cu_seqlens"] = torch.cat([lens_d.new_zeros(1), lens_d.cumsum(0)]).to(torch.int32)
        s["total"] = int(lens.sum())
        return s
    s["q"] = torch.randn(case["batch"], case["hq"], d, generator=g, device=DEV, dtype=BF16)
    s["kv_lens"] = lens_d.to(torch.int32)
    s["kv_starts"] = (lens_d - case["window"]).clamp(min=0).to(torch.int32) if case["window"] else None
    s["sink"] = torch.randn(case["hq"], generator=g, device=DEV) if case["sink"] else None
    s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

EPS = 1e-6


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import flexible_mask_flashattention_gb300 as ffa
    op = s["case"]["op"]
    if op == "norm":
        return ffa.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"], eps=EPS,
                                interleaved=s["case"]["interleaved"])
    if op == "norm_bwd":
        return ffa.qk_norm_rope_bwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"],
                                    s["dq_out"], s["dk_out"], eps=EPS, interleaved=s["case"]["interleaved"])
    if op in ("write", "write_step"):
        ffa.kv_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        return s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"]
    if op == "read":
        return ffa.kv_cache_read(s["k_cache"], s["v_cache"], s["page_table"], s["cu_seqlens"], s["total"],
                                 k_exp=s["k_exp"], v_exp=s["v_exp"])
    return ffa.fwd_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["scale"],
                          k_exp=s["k_exp"], v_exp=s["v_exp"], kv_starts=s["kv_starts"], sink=s["sink"])


def _pairs(x, rot, interleaved):
    """The two halves of the rotated columns' pairs, and the columns behind them."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    return a, b, x[..., rot:]


def _unpairs(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _cos_sin(s):
    cs = s["table"][s["positions"].long()][:, None, :]
    half = s["case"]["rot"] // 2
    return cs[..., :half], cs[..., half:]


def _norm_rope(s, x, w):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    cos, sin = _cos_sin(s)
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a, b, rest = _pairs(y, rot, inter)
    return _unpairs(a * cos - b * sin, b * cos + a * sin, rest, inter).to(BF16)


def _norm_rope_bwd(s, x, w, dout):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    cos, sin = _cos_sin(s)
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    a, b, rest = _pairs(dout.float(), rot, inter)
    dy = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, inter)
    dw = (dy * xh).sum((0, 1))
    dy = dy * w
    return (r * (dy - xh * (dy * xh).mean(-1, keepdim=True))).to(BF16), dw


def _pow2(n):
    """2^n in 32 bits, exactly, for -126 <= n <= 127."""
    return ((n.int() + 127) << 23).view(F32)


def _quantise(x):
    """e4m3 codes and exponent bytes of rows: x = code * 2^(byte - 127), the smallest such scale that holds the row."""
    x = x.float()
    f, e = torch.frexp(x.abs().amax(-1))
    n = torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-126)
    return (x * _pow2(-n)[..., None]).to(FP8), (n + 127).to(torch.uint8)


def _stored(x, exps):
    return x.float() if exps is None else x.float() * _pow2(exps.int() - 127)[..., None]


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _norm_rope(s, s["q"], s["q_weight"]), _norm_rope(s, s["k"], s["k_weight"])
    if op == "norm_bwd":
        dq, dqw = _norm_rope_bwd(s, s["q"], s["q_weight"], s["dq_out"])
        dk, dkw = _norm_rope_bwd(s, s["k"], s["k_weight"], s["dk_out"])
        return dq, dk, dqw, dkw
    page = s["case"]["page"]
    if op in ("write", "write_step"):
        at, off = s["slots"] // page, s["slots"] % page
        for x, cache, exps in ((s["k"], s["k_cache"], s["k_exp"]), (s["v"], s["v_cache"], s["v_exp"])):
            if exps is None:
                cache[at, :, off] = x
            else:
                codes, e = _quantise(x)
                cache.view(torch.uint8)[at, :, off] = codes.view(torch.uint8)
                exps[at, :, off] = e
        return s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"]
    if op == "read":
        cu = s["cu_seqlens"].long()
        row = torch.arange(s["total"], device=DEV)
        seq = torch.searchsorted(cu, row, right=True) - 1
        pos = row - cu[seq]
        at, off = s["page_table"][seq, pos // page].long(), pos % page
        return tuple(_stored(c.view(torch.uint8)[at, :, off].view(FP8) if e is not None else c[at, :, off],
                             None if e is None else e[at, :, off]).to(BF16)
                     for c, e in ((s["k_cache"], s["k_exp"]), (s["v_cache"], s["v_exp"])))
    q = s["q"].float()
    b, hq, d = q.shape
    table = s["page_table"].clamp(min=0).long()
    hkv = s["case"]["hkv"]

    def padded(c, e):   # [b, hkv, keys, d] of every sequence's pages
        x = c.view(torch.uint8)[table].view(FP8) if e is not None else c[table]
        return _stored(x, None if e is None else e[table]).transpose(1, 2).reshape(b, hkv, -1, d)

    k = padded(s["k_cache"], s["k_exp"])
    logits = torch.matmul(q.view(b, hkv, -1, d), k.transpose(-1, -2)).mul_(s["scale"])
    del k
    j = torch.arange(logits.shape[-1], device=DEV)
    keep = j[None, :] < s["kv_lens"][:, None]
    if s["kv_starts"] is not None:
        keep &= j[None, :] >= s["kv_starts"][:, None]
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
    v = torch.where(keep.transpose(-1, -2), padded(s["v_cache"], s["v_exp"]), 0.0)
    out = torch.matmul(p, v) / total
    lse = (m + torch.log(total)).view(b, hq).t().contiguous()
    return out.view(b, hq, d).to(BF16), lse


# ---- the same in 64 bits, from the definitions ----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("norm", "norm_bwd"):
            return _exact_norm(s)
        if op in ("write", "write_step"):
            return _exact_write(s)
        return _exact_read(s) if op == "read" else _exact_decode(s)


def _exact_matrix(s, rows):
    """The rotation of each of `rows` as a dense matrix [n, d, d] in 64 bits."""
    d, rot = s["case"]["d"], s["case"]["rot"]
    i = torch.arange(rot // 2, device=DEV)
    a, b = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + rot // 2)
    cs = s["table"].to(F64)[s["positions"][rows].long()]
    m = torch.eye(d, dtype=F64, device=DEV).repeat(len(cs), 1, 1)
    m[:, a, a] = cs[:, :rot // 2]
    m[:, b, b] = cs[:, :rot // 2]
    m[:, a, b] = -cs[:, rot // 2:]
    m[:, b, a] = cs[:, rot // 2:]
    return m


def _exact_norm(s):
    """out = M diag(w) x / |x|rms, with M the position's rotation matrix; gradients by the chain rule through M, w and the norm."""
    t, d, back = s["case"]["tokens"], s["case"]["d"], s["case"]["op"] == "norm_bwd"
    outs, dws = [], []
    for name in ("q", "k"):
        x_all, w = s[name], s[name + "_weight"].to(F64)
        parts, dw = [], torch.zeros(d, dtype=F64, device=DEV)
        for i in range(0, t, 4096):
            rows = slice(i, min(t, i + 4096))
            m = _exact_matrix(s, rows)
            x = x_all[rows].to(F64)
            rms = (torch.einsum("thd,thd->th", x, x) / d + EPS).sqrt()[..., None]
            if not back:
                parts.append(torch.bmm(w * (x / rms), m.transpose(1, 2)))
                continue
            g = torch.bmm(s["d" + name + "_out"][rows].to(F64), m)
            dw += torch.einsum("thd,thd->d", g, x / rms)
            g = g * w
            parts.append(g / rms - x * torch.einsum("thd,thd->th", g, x)[..., None] / (d * rms ** 3))
        outs.append(torch.cat(parts))
        dws.append(dw)
    return tuple(outs + dws) if back else tuple(outs)


E4M3_VALUES = sorted({(m / 8.0 + (1 if e else 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)
                      if (e, m) != (15, 7)})


def _power(n):
    """2^n in 64 bits, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(F64)


def _nearest_e4m3(x):
    """The nearest of the e4m3 values, ties to the even code."""
    grid = torch.tensor(E4M3_VALUES, dtype=F64, device=DEV)
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.sign(x) * torch.where(up, grid[hi], grid[lo])


def _exact_write(s):
    page = s["case"]["page"]
    outs, exps = [], []
    for n in "kv":
        cache = torch.zeros(s[n + "_cache"].shape, dtype=F64, device=DEV)
        e_all = None if s[n + "_exp"] is None else torch.zeros(s[n + "_exp"].shape, dtype=torch.uint8, device=DEV)
        for i in range(0, len(s["slots"]), 32768):
            x, slots = s[n][i:i + 32768].to(F64), s["slots"][i:i + 32768]
            if e_all is not None:
                top = x.abs().max(-1).values
                e = torch.full_like(top, -126.0)
                some = top > 0
                e[some] = torch.ceil(torch.log2(top[some] / 448.0))
                e = torch.where(top <= 448.0 * _power(e - 1), e - 1, torch.where(top > 448.0 * _power(e), e + 1, e)).clamp(min=-126)
                e_all[slots // page, :, slots % page] = (e + 127).to(torch.uint8)
                x = _nearest_e4m3(x / _power(e)[..., None])
            cache[slots // page, :, slots % page] = x
        outs.append(cache)
        exps.append(e_all)
    return tuple(outs + exps)


def _exact_rows(s, n, b, lo, hi):
    """Rows [lo, hi) of sequence b in 64 bits: [keys, hkv, d]."""
    page = s["case"]["page"]
    pages = s["page_table"][b, lo // page:(hi + page - 1) // page].long()
    first = lo - lo // page * page
    x = s[n + "_cache"].view(torch.uint8)[pages].view(FP8) if s[n + "_exp"] is not None else s[n + "_cache"][pages]
    x = x.to(F64)
    if s[n + "_exp"] is not None:
        x = x * _power(s[n + "_exp"][pages].to(torch.int64) - 127)[..., None]
    return x.transpose(1, 2).flatten(0, 1)[first:first + hi - lo]


def _exact_read(s):
    cu = s["cu_seqlens"].tolist()
    return tuple(torch.cat([_exact_rows(s, n, b, 0, cu[b + 1] - cu[b]) for b in range(len(cu) - 1)]) for n in "kv")


def _exact_decode(s):
    case = s["case"]
    lens, hkv, d = s["kv_lens"].tolist(), case["hkv"], case["d"]
    starts = s["kv_starts"].tolist() if s["kv_starts"] is not None else [0] * len(lens)
    outs, lses = [], []
    for b, (lo, hi) in enumerate(zip(starts, lens)):
        q = s["q"][b].to(F64).view(hkv, -1, d)
        z = torch.einsum("hgd,khd->hgk", q, _exact_rows(s, "k", b, lo, hi)) * s["scale"]
        if s["sink"] is not None:
            z = torch.cat([z, s["sink"].to(F64).view(hkv, -1, 1)], -1)
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - lse[..., None])[..., :hi - lo]
        outs.append(torch.einsum("hgk,khd->hgd", p, _exact_rows(s, "v", b, lo, hi)).reshape(-1, d))
        lses.append(lse.reshape(-1))
    return torch.stack(outs), torch.stack(lses, 1)
