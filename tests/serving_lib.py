"""What the tests of the paged cache's types share: caches of every type, what they hold, and one-token attention against the oracle.

Tolerance of one-token attention (u = 2^-24, a bf16 rounding is off by at most 2^-8 of the value), mass = sum_j p_j |v_j|,
delta = (d + 16) u max_j sum_i |scale q_i k_ji| the scores' error (32-bit products and sums, factors of the scale):
  out  2^-8 |ref|                 the bf16 output
       (rho + 2 delta + acc) mass rho the rounding of a weight (2^-16 as a bf16 pair, 2^-11 + 2^-15 as f16 with its exponent's additions), acc =
                                  (keys / 16 + 32) 2^-22 the accumulation's and the exponentials'
       keys 2^-33 max|v|          quantised types: an f16 weight below the normal range is off by 2^-25 at most, the largest is held as 2^10 at
                                  least, a code (times its scale) is 2688 2^n at most, and the row of the largest weight has one
                                  of 1344 (1 - 2^-4) 2^n: 2^-35 times 2.14 max|v| a key (e4m3: 448 and 224, times 2)
  lse  delta + 2^-20 + 4 u |lse|
"""
import numpy as np

from oracle import serving as S
from test_gpu_serving import U, bits, f64

KINDS = ("bf16", "e4m3", "e2m1")


class Cache:
    """k and v [pages, hkv, page, d] of one type, on the GPU, all zeros (or `fill` bytes)."""

    def __init__(self, pages, hkv, page, d, kind, fill=0):
        import torch
        self.kind, self.shape = kind, (pages, hkv, page, d)
        z = lambda dtype, last: torch.full((pages, hkv, page) + last, fill, dtype=torch.uint8, device="cuda").view(dtype)  # noqa: E731
        for n in "kv":
            if kind == "bf16":
                setattr(self, n, z(torch.bfloat16, (2 * d,)))
            elif kind == "e4m3":
                setattr(self, n, z(torch.float8_e4m3fn, (d,)))
            else:
                setattr(self, n, z(torch.uint8, (d // 2,)))
            setattr(self, n + "_exp", None if kind == "bf16" else z(torch.uint8, ()))
            setattr(self, n + "_scale", z(torch.float8_e4m3fn, (d // 16,)) if kind == "e2m1" else None)

    def more(self):
        return {n: getattr(self, n) for n in ("k_exp", "v_exp", "k_scale", "v_scale")}

    def arrays(self):
        """Every array as bytes [pages, hkv, page, ...], by name; copies."""
        out = {}
        for n in "kv":
            for part in ("", "_exp", "_scale"):
                x = getattr(self, n + part)
                if x is not None:
                    out[n + part] = bits(x).reshape(self.shape[:3] + (-1,)).copy()
        return out

    def values(self, n):
        """What k or v holds, in 64 bits."""
        pages, hkv, page, d = self.shape
        x, e, s = (getattr(self, n + part) for part in ("", "_exp", "_scale"))
        if self.kind == "bf16":
            return f64(x)
        if self.kind == "e4m3":
            return S.stored_values(bits(x).reshape(self.shape), e.cpu().numpy())
        return S.stored_values4(bits(x).reshape(pages, hkv, page, d // 2), bits(s).reshape(pages, hkv, page, d // 16), e.cpu().numpy())

    def expect(self, want, n, x, slots):
        """Into the arrays `want`, what writing rows x [tokens, hkv, d] (64 bits) at slots leaves, by the oracle."""
        pages, hkv, page, d = self.shape
        for i, slot in enumerate(slots):
            if not 0 <= slot < pages * page:
                continue
            at = (slot // page, slice(None), slot % page)
            for h in range(hkv):
                where = (at[0], h, at[2])
                if self.kind == "bf16":
                    import torch
                    want[n][where] = torch.from_numpy(x[i, h]).bfloat16().view(torch.uint8).numpy()
                elif self.kind == "e4m3":
                    want[n][where], want[n + "_exp"][where] = S.quantise_row(x[i, h])
                else:
                    codes, want[n + "_scale"][where], want[n + "_exp"][where] = S.quantise_row4(x[i, h])
                    want[n][where] = S.packed_codes(codes)


def same_arrays(got, want):
    for n in want:
        assert np.array_equal(got[n], want[n]), (n, np.argwhere(got[n] != want[n])[:5])


def problem(lens, hq, hkv, d, page, kind, seed, spread=0.5, extra_pages=2):
    """A written cache, its page table, queries and lengths, as keyword arguments of fwd_decode, and the Cache."""
    import flexible_mask_flashattention_gb300 as m
    import torch
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-n // page)) for n in lens]
    pages, width = sum(need) + extra_pages, max(1, max(need, default=1))
    c = Cache(pages, hkv, page, d, kind)
    n = pages * page
    k = torch.randn(n, hkv, d, generator=g).bfloat16().cuda()
    v = (torch.randn(n, hkv, d, generator=g) * torch.exp(spread * torch.randn(n, hkv, 1, generator=g))).bfloat16().cuda()
    m.kv_cache_write(k, v, c.k, c.v, torch.arange(n, device="cuda"), **c.more())
    order, table, used = torch.randperm(pages, generator=g).int(), torch.full((len(lens), width), -1, dtype=torch.int32), 0
    for b, count in enumerate(need):
        table[b, :count] = order[used:used + count]
        used += count
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16().cuda()
    return dict(q=q, k_cache=c.k, v_cache=c.v, page_table=table.cuda(), kv_lens=torch.tensor(lens, dtype=torch.int32).cuda(), **c.more()), c


def check_decode(out, lse, p, cache, scale, starts=None, firsts=None, sink=None, skip=()):
    kv, vv = cache.values("k"), cache.values("v")
    d = p["q"].shape[-1]
    q, lens, table, got, gl = f64(p["q"]), p["kv_lens"].cpu().numpy(), p["page_table"].cpu().numpy(), f64(out), f64(lse)
    sk = None if sink is None else f64(sink)
    for b in range(len(lens)):
        if b in skip:
            continue
        keys = S.visible_keys(int(lens[b]), 0 if starts is None else int(starts[b]), 0 if firsts is None else int(firsts[b]))
        vb = S.gather_keys(vv, table[b], keys)
        ro, rl, mass, size = S.decode(q[b], S.gather_keys(kv, table[b], keys), vb, scale, sk)
        delta = (d + 16) * U * size
        rho = 2.0 ** -16 if cache.kind == "bf16" else 2.0 ** -11 + 2.0 ** -15
        w = rho + 2 * delta + (len(keys) / 16 + 32) * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ro) + w[:, None] * mass + 1e-30
        if cache.kind != "bf16":
            tol = tol + len(keys) * 2.0 ** -33 * np.abs(vb).max(initial=0.0)
        err = np.abs(got[b] - ro)
        assert (err <= tol).all(), (b, len(keys), (err / tol).max())
        fin = np.isfinite(rl)
        assert np.array_equal(gl[:, b][~fin], rl[~fin]), b
        el = np.abs(gl[:, b][fin] - rl[fin])
        assert (el <= delta[fin] + 2.0 ** -20 + 4 * U * np.abs(rl[fin])).all(), (b, el.max())
