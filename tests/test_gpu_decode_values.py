"""e4m3 one-token attention over value rows of very different sizes, against the fp64 oracle, with a tolerance that counts what a
row weighs: a row that is large but has no weight for a query must not cost that query's other keys their bits.

Tolerance of an output, from the roundings on its way (u = 2^-24):
  2^-8 |ref|                    the bf16 output
  (2^-11 + 2^-15) mass          mass = sum_j p_j |v_j|.  A weight e^{s_j} 2^{n_j} is an f16 value (2^-11); its exponent s_j log2(e) + n_j - ref is
                                two fp32 additions of terms up to 2^7 beside the score's own: 2 u 2^8 ln 2 < 2^-15
  (2 delta + acc) mass          delta = (d + 16) u max_j sum_i |scale q_i k_ji| the scores' error, acc = (keys / 16 + 32) 2^-22 the
                                accumulation's
  keys 2^-34 max_j p_j |v_j|    a weight under f16's normal range is off by at most 2^-25 where the query's largest is held as 2^10 at least;
                                codes reach 448 in the one row and lie over 224 somewhere in the other: 2^-35 448 / 224 a key
"""
import numpy as np
import pytest

from oracle import serving as S
from test_gpu_serving import U, cache_values, f64, ffa, ffa_write, new_cache  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


def problem(n, group, d, ratio_log2, where, seed):
    """One sequence of n keys, one kv head.  Rows of V that are `where` are 2^ratio_log2 times the others; column 0 of K is -1 for those
    and 0 for the rest, so that a query's column 0 decides what they weigh."""
    import torch
    r = np.random.default_rng(seed)
    page = 64
    pages = -(-n // page)
    big = {"first": np.arange(n) < 40, "last": np.arange(n) >= n - 40, "mixed": r.random(n) < 0.3,
           "one": np.arange(n) == n // 2}[where]
    v = r.normal(size=(pages * page, 1, d))
    v[:n][big] *= 2.0 ** ratio_log2
    k = np.zeros((pages * page, 1, d))
    k[:n, 0, 0] = np.where(big, -1.0, 0.0)
    k[:, 0, 1:] = r.normal(size=(pages * page, d - 1))
    q = 0.05 * r.normal(size=(1, group, d))
    # weights of the large rows against the others': e^0, then so little that they count as much as, and far less than, the rest
    at = np.array([0.0, ratio_log2 * np.log(2.0), 2.0 * ratio_log2 * np.log(2.0) + 20.0, 400.0])
    q[0, :, 0] = at[np.arange(group) % 4]
    kc, vc, ke, ve = new_cache(pages, 1, page, d, True)
    t = [torch.tensor(x).bfloat16().cuda() for x in (q, k, v)]
    ffa_write(t[1], t[2], kc, vc, ke, ve)
    return dict(q=t[0], k_cache=kc, v_cache=vc, page_table=torch.arange(pages, dtype=torch.int32).cuda()[None],
                kv_lens=torch.tensor([n], dtype=torch.int32).cuda(), k_exp=ke, v_exp=ve)


def check(out, lse, p, scale, lens):
    kv, vv = cache_values(p)
    d, table, q, got, gl = p["q"].shape[-1], p["page_table"].cpu().numpy(), f64(p["q"]), f64(out), f64(lse)
    hq, hkv = q.shape[1], kv.shape[1]
    for b, n in enumerate(lens):
        kb, vb = S.gather_rows(kv, table[b], 0, n), S.gather_rows(vv, table[b], 0, n)
        ro, rl, mass, size = S.decode(q[b], kb, vb, scale)
        row = np.abs(vb).max(-1)                                                  # [keys, hkv]
        top = np.array([(np.exp(scale * kb[:, h // (hq // hkv)] @ q[b, h] - rl[h]) * row[:, h // (hq // hkv)]).max() for h in range(hq)])
        delta = (d + 16) * U * size
        w = 2.0 ** -11 + 2.0 ** -15 + 2 * delta + (n / 16 + 32) * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ro) + w[:, None] * mass + n * 2.0 ** -34 * top[:, None]
        err = np.abs(got[b] - ro)
        assert (err <= tol).all(), (b, n, (err / tol).max(-1))
        assert (np.abs(gl[:, b] - rl) <= delta + 2.0 ** -20 + 4 * U * np.abs(rl)).all()


@pytest.mark.parametrize("where", ["first", "last", "mixed", "one"])
@pytest.mark.parametrize("ratio_log2", [12, 24, 28, 40, 100])
@pytest.mark.parametrize("n,group,d", [(700, 4, 128), (700, 4, 64), (700, 12, 128), (700, 12, 64), (50000, 4, 64), (50000, 12, 128)])
def test_large_value_rows_without_weight(ffa, n, group, d, ratio_log2, where):
    p = problem(n, group, d, ratio_log2, where, n + group + d + ratio_log2)
    check(*ffa.fwd_decode(**p, scale=1.0), p, 1.0, [n])


def test_values_at_both_ends_of_the_range(ffa):
    """All rows tiny, all rows huge, and an exponent byte of 0, which stands for zeros."""
    import torch
    for mag in (2.0 ** -110, 2.0 ** -60, 2.0 ** 60, 2.0 ** 110):
        p = problem(300, 4, 64, 0, "mixed", 3)
        v = torch.tensor(np.random.default_rng(4).normal(size=(320, 1, 64)) * mag).bfloat16().cuda()
        k = torch.tensor(np.random.default_rng(5).normal(size=(320, 1, 64))).bfloat16().cuda()
        ffa_write(k, v, p["k_cache"], p["v_cache"], p["k_exp"], p["v_exp"])
        check(*ffa.fwd_decode(**p, scale=0.1), p, 0.1, [300])
        p["v_exp"][1:3] = 0
        check(*ffa.fwd_decode(**p, scale=0.1), p, 0.1, [300])
    p["v_exp"][:] = 0
    out, lse = ffa.fwd_decode(**p, scale=0.1)
    assert (out == 0).all() and lse.isfinite().all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [4, 10, 14, 17, 20, 23])
def test_one_key_with_a_large_score(ffa, power, sign):
    """A row of one key is its value, whatever its score: the scores lie next to a power of two (in log2 units), where the value's
    exponent, added to them, changes their rounding.  f16 weight and its exponent's additions, bf16 output."""
    import torch
    d, n = 64, 64
    g = torch.Generator().manual_seed(power)
    k, q = torch.zeros(n * 16, 1, d), torch.zeros(n, 3, d)
    k[:, 0, 0], q[:, :, 0] = 1.0, 1.0
    v = torch.randn(n * 16, 1, d, generator=g) * 2.0 ** torch.linspace(-70, 70, n).repeat_interleave(16)[:, None, None]
    kc, vc, ke, ve = new_cache(n, 1, 16, d, True)
    ffa_write(k.bfloat16().cuda(), v.bfloat16().cuda(), kc, vc, ke, ve)
    p = dict(q=q.bfloat16().cuda(), k_cache=kc, v_cache=vc, page_table=torch.arange(n, dtype=torch.int32).cuda()[:, None],
             kv_lens=torch.ones(n, dtype=torch.int32).cuda(), k_exp=ke, v_exp=ve)
    for off in (-40.3, -3.7, 0.4, 33.9):
        score = sign * (2.0 ** power + off)
        out, lse = ffa.fwd_decode(**p, scale=score * float(np.log(2.0)))
        want = cache_values(p)[1][:, :, 0]
        assert (np.abs(f64(out) - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15) * np.abs(want)).all()
        ref = score * np.log(2.0)
        assert (np.abs(f64(lse) - ref) <= 2.0 ** -20 + 8 * U * abs(ref)).all()
