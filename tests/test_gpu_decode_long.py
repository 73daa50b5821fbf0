"""One-token attention where every CTA walks over several blocks of a unit, against the fp64 oracle: later blocks of a unit (the ring filled
again, references raised while sums and outputs are non-zero), shares that begin and end inside units, units that a CTA opens behind the
end of another, and joins of more parts than one round takes.  Lengths follow the device's SM count, and each case asserts on the host,
from the shares' arithmetic, that it holds what it is for.

Scores rise or fall along the sequence by up to 200, differently for each head, and the value rows grow by 2^20, so that the keys that
matter are the last ones, the first ones, or all of them, weighed against the values' growth.

Tolerance (u = 2^-24), mass = sum_j p_j |v_j|, delta = (d + 16) u max_j sum_i |scale q_i k_ji|:
  out  2^-8 |ref|                   the bf16 output
       (rho + 2 delta + acc) mass   rho 2^-16 for weights as bf16 pairs; 2^-11 + 2^-15 for f16 weights and their exponents' additions.  acc = (keys / 16 +
                                    32) 2^-22 the accumulation's; raising a reference costs 2^-22 of what was summed before it, which is then
                                    2^-5 of the rest at most, so all of them cost less than one more 2^-21 (in acc's 32)
       keys 2^-34 max_j p_j |v_j|   e4m3: f16 weights under the normal range, relative to the query's largest
  lse  delta + 2^-20 + 4 u |lse|
"""
import numpy as np
import pytest

from oracle import serving as S
from test_gpu_serving import U, bits, cache_values, f64, ffa, ffa_write, new_cache  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


def block_of(d, fp8, group):
    """(keys of a strip, of a block) of the kernel that takes this configuration, and its units a kv head."""
    tiles = 2 if group > 8 else 1
    strip = 16 if d == 128 and not fp8 else 32
    return strip, strip * (8 if tiles == 2 or d == 128 else 12), -(-group // (8 * tiles))


def shares(lens, starts, units, strip, block, ctas):
    """What each CTA's share of the block list holds: a list of parts (unit, blocks, from its start, to its end, slot)."""
    per = []
    for n, s in zip(lens, starts):
        n = max(0, n)
        s = min(max(0, s), n)
        per += [max(1, -(-(n - s // strip * strip) // block))] * units
    ends, total = np.cumsum(per), sum(per)
    parts = min(total, ctas)
    out = []
    for c in range(parts):
        t, t1, mine = total * c // parts, total * (c + 1) // parts, []
        while t < t1:
            u = int(np.searchsorted(ends, t, side="right"))
            first, stop = int(ends[u]) - per[u], min(t1, int(ends[u]))
            mine.append((u, stop - t, t == first, stop == ends[u], 2 * c + (1 if mine else 0)))
            t = stop
        out.append(mine)
    return out


def problem(lens, hq, hkv, d, fp8, seed, page=64):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-max(0, n) // page) for n in lens]
    pages, width = sum(need) + 1, max(need)
    kc, vc, ke, ve = new_cache(pages, hkv, page, d, fp8)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    k = torch.zeros(pages * page, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    used = 0
    for b, n in enumerate(lens):
        ids = order[used:used + need[b]]
        table[b, :need[b]], used = ids, used + need[b]
        if n <= 0:
            continue
        j = torch.arange(n, device="cuda")
        rows = ids.long()[j // page] * page + j % page
        along = (j.double() / max(1, n - 1))[:, None, None]
        kb = torch.randn(n, hkv, d, generator=g, device="cuda", dtype=torch.float64)
        kb[:, :, :1] = along
        vb = torch.randn(n, hkv, d, generator=g, device="cuda", dtype=torch.float64) * 2.0 ** (20 * along)
        k[rows], v[rows] = kb.bfloat16(), vb.bfloat16()
    ffa_write(k, v, kc, vc, ke, ve)
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda")
    slopes = torch.tensor([0.0, 8.0, 40.0, 200.0, -14.0, -100.0], device="cuda")
    q[:, :, 0] = slopes[torch.arange(hq, device="cuda") % 6] * d ** 0.5
    return dict(q=q.bfloat16(), k_cache=kc, v_cache=vc, page_table=table, kv_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                k_exp=ke, v_exp=ve)


def check(out, lse, p, scale, lens, starts, sink):
    kv, vv = cache_values(p)
    fp8, d, table, q, got, gl = p["k_exp"] is not None, p["q"].shape[-1], p["page_table"].cpu().numpy(), f64(p["q"]), f64(out), f64(lse)
    group = q.shape[1] // kv.shape[1]
    for b, (n, s) in enumerate(zip(lens, starts)):
        n = max(0, n)
        s = min(max(0, s), n)
        kb, vb = S.gather_rows(kv, table[b], s, n), S.gather_rows(vv, table[b], s, n)
        ro, rl, mass, size = S.decode(q[b], kb, vb, scale, sink)
        delta = (d + 16) * U * size
        w = (2.0 ** -11 + 2.0 ** -15 if fp8 else 2.0 ** -16) + 2 * delta + ((n - s) / 16 + 32) * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ro) + w[:, None] * mass + 1e-30
        if fp8 and n > s:
            row = np.abs(vb).max(-1)
            tol += (n - s) * 2.0 ** -34 * np.array([(np.exp(scale * kb[:, h // group] @ q[b, h] - rl[h]) * row[:, h // group]).max()
                                                    for h in range(q.shape[1])])[:, None]
        err = np.abs(got[b] - ro)
        assert (err <= tol).all(), (b, n, s, (err / tol).max(-1))
        fin = np.isfinite(rl)
        assert np.array_equal(gl[:, b][~fin], rl[~fin]), b
        assert (np.abs(gl[fin, b] - rl[fin]) <= (delta + 2.0 ** -20 + 4 * U * np.abs(rl))[fin]).all(), (b, n, s)


CASES = [("ragged", 8, 2), ("ragged", 3, 1), ("many", 6, 2), ("many", 24, 2), ("single", 4, 1), ("single", 12, 1), ("single", 40, 1)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind,hq,hkv", CASES)
def test_decode_over_several_blocks_a_cta(ffa, kind, hq, hkv, d, fp8):
    import torch
    sms = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    strip, block, subs = block_of(d, fp8, hq // hkv)
    keys = int((5.3 if kind != "many" else 4.2) * sms * block / (hkv * subs))
    r = np.random.default_rng(hq + d)
    if kind == "single":
        lens, starts = [keys], [0]
    elif kind == "ragged":
        lens = [int(keys * f) for f in (0.36, 0.0, 0.21, 0.29)] + [1, int(keys * 0.2)]
        starts = [0, 0, 77, 5, 0, int(keys * 0.2) - 3 * block - 11]
    else:
        f = r.dirichlet(np.full(41, 0.35))
        lens = [int(keys * x) for x in f]
        starts = [0 if i % 3 else int(r.integers(0, 50)) for i in range(41)]
    split = shares(lens, starts, hkv * subs, strip, block, sms)
    assert max(part[1] for mine in split for part in mine) >= 4, "no CTA walks several blocks of a unit"
    opened = [part for mine in split for part in mine if part[2] and not part[3]]
    if kind != "single":
        assert any(part[4] % 2 for part in opened), "no unit is opened behind the end of another"
        assert any(not mine[0][2] and mine[0][3] for mine in split), "no share begins inside a unit that ends in it"
    else:
        parts = np.bincount([part[0] for mine in split for part in mine])
        assert parts.max() > (32 if d == 128 else 64) or subs > 1, "one round of the join is enough"
    p = problem(lens, hq, hkv, d, fp8, hq * 1000 + d + len(lens))
    scale, st = d ** -0.5, torch.tensor(starts, dtype=torch.int32).cuda()
    sink = torch.linspace(-4, 9, hq).cuda() if kind == "ragged" else None
    out, lse = ffa.fwd_decode(**p, scale=scale, kv_starts=st, sink=sink)
    check(out, lse, p, scale, lens, starts, None if sink is None else f64(sink))
    again, la = ffa.fwd_decode(**p, scale=scale, kv_starts=st, sink=sink)
    assert (bits(again) == bits(out)).all() and (bits(la) == bits(lse)).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_bad_page_and_a_bad_length_in_a_long_batch(ffa, fp8):
    """In a batch whose units are split over CTAs, the rows of one sequence are NaN and the others' keep every bit."""
    import torch
    p = problem([40000, 30000, 1, 50000], 6, 2, 128, fp8, 5)
    good, gl = ffa.fwd_decode(**p, scale=0.1)
    p["page_table"][1, 444] = -1                                   # in a middle block of a unit
    p["kv_lens"][2] = p["page_table"].shape[1] * 64 + 1            # one key more than its row of pages holds: one block, as before
    out, lse = ffa.fwd_decode(**p, scale=0.1)
    for b in (0, 3):
        assert (bits(out[b]) == bits(good[b])).all() and (bits(lse[:, b]) == bits(gl[:, b])).all()
    for b in (1, 2):
        assert out[b].isnan().all() and lse[:, b].isnan().all()
