"""GPU parity of qk_norm_rope(_bwd), kv_cache_write / kv_cache_read and fwd_decode against the fp64 oracle
(oracle/serving.py), at the sizes, masks and values where they can go wrong.

Tolerances, from the roundings a result goes through (u = 2^-24, half a step of fp32; a bf16 rounding is off by at most 2^-8
of the value):
  norm/rope out   2^-8 |ref| + 32 u max|y|: one bf16 rounding; about 10 fp32 roundings of terms no larger than the row's largest, the
                  sum of squares' included (its 7 sequential and 4 tree adds act on the root, halved), rsqrtf 2 ulp
  dx              2^-8 |ref| + 64 u r (max|h| + max|x| |c|): two such sums, h x and x^2
  dweight         (depth + 24) u sum|terms|: depth the longest chain of fp32 adds
  cache           bit-exact codes and bytes; reading back exact
  decode          2^-8 |ref| + (rho + 2 delta + acc) sum_j p_j |v_j|, with delta = (d + 16) u max_j sum_i |scale q_i k_ji|
                  the scores' error (32-bit products and sums, factors of the scale), rho the rounding of a weight (2^-16 as a bf16
                  pair, 2^-11 as f16), acc = (keys / 16 + 32) 2^-22 the accumulation's (tensor-core adds
                  may truncate) and the exponentials' (2^-22)
                  and, for e4m3, + keys 2^-34 max|v|: an f16 weight below its normal range is off by at most 2^-25, and the largest weight is
                  held as 2^10 at least, relative to a scale whose codes reach 448 > max|v| / 2 of the row it is of: 2^-35 times
                  2 max|v| a key (seen where the keys that matter have a zero in a column)
  lse             delta + 2^-20 + 4 u |lse|
"""
import numpy as np
import pytest

import oracle as O
from oracle import serving as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ffa():
    import torch
    assert torch.cuda.is_available()
    import __graft_entry__
    __graft_entry__.build()
    import flexible_mask_flashattention_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    import torch
    return t.detach().contiguous().view(torch.uint8).cpu().numpy()


# ---- norm and rotation -----------------------------------------------------------------------------------------------

def rope_table(max_pos, rot):
    import torch
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([ang.cos(), ang.sin()], 1).float().cuda()


def norm_inputs(tokens, hq, hkv, d, rot, seed, max_pos=500, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(tokens, hq + 2 * hkv, d, generator=g) * scale).bfloat16().cuda()
    pos = torch.randint(0, max_pos, (tokens,), generator=g, dtype=torch.int32).cuda()
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    dout = [torch.randn(tokens, h, d, generator=g).bfloat16().cuda() for h in (hq, hkv)]
    return qkv[:, :hq], qkv[:, hq:hq + hkv], w[0], w[1], rope_table(max_pos, rot), pos, dout[0], dout[1]


def check_norm(out, x, w, table, pos, eps, inter):
    ref = S.norm_rope(f64(x), f64(w), f64(table), pos.cpu().numpy(), eps, inter)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fin = ~np.isnan(ref)
    x, w = f64(x), f64(w)
    y = np.abs(x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w).max(-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(ref) + 32 * U * y
    assert (np.abs(got - ref) <= tol)[fin].all(), np.nanmax(np.abs(got - ref) / tol)


NORM_CASES = [(1, 1, 1, 64, 64, False), (1, 16, 4, 128, 128, False), (3, 3, 3, 128, 16, False), (37, 6, 2, 64, 32, True),
              (130, 5, 1, 128, 48, False), (65, 9, 3, 64, 48, True), (257, 64, 8, 128, 128, True), (1000, 17, 17, 64, 64, False),
              (2049, 2, 1, 128, 96, True)]


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter", NORM_CASES)
def test_norm_rope(ffa, tokens, hq, hkv, d, rot, inter):
    q, k, qw, kw, t, pos, _, _ = norm_inputs(tokens, hq, hkv, d, rot, tokens + hq)
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos, eps=1e-5, interleaved=inter)
    check_norm(qo, q, qw, t, pos, 1e-5, inter)
    check_norm(ko, k, kw, t, pos, 1e-5, inter)
    qc, kc = ffa.qk_norm_rope(q.contiguous(), k.contiguous(), qw, kw, t, pos, eps=1e-5, interleaved=inter)
    assert (bits(qc) == bits(qo)).all() and (bits(kc) == bits(ko)).all()   # strided or not, the same


def check_norm_bwd(ffa, grads, q, k, qw, kw, t, pos, dqo, dko, eps, inter):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    d = q.shape[-1]
    for dx, dw, x, w, dout in ((grads[0], grads[2], q, qw, dqo), (grads[1], grads[3], k, kw, dko)):
        x64, w64, g64, p = f64(x), f64(w), f64(dout), pos.cpu().numpy()
        rx, rw, mass = S.norm_rope_grad(x64, w64, f64(t), p, g64, eps, inter)
        r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
        h = np.sqrt(2) * np.abs(g64).max(-1, keepdims=True) * np.abs(w64).max()
        c = r ** 2 * h * np.abs(x64).mean(-1, keepdims=True)
        tol = 2.0 ** -8 * np.abs(rx) + 64 * U * r * (h + np.abs(x64).max(-1, keepdims=True) * c)
        err = np.abs(f64(dx) - rx)
        assert (err <= tol).all(), (err / tol).max()
        rows = x.shape[0] * ((q.shape[1] + k.shape[1]) * d // 512 + 2)
        depth = 2 * (rows / (8 * sms) + 1) + 64
        errw = np.abs(f64(dw) - rw)
        assert (errw <= (depth + 24) * U * mass + 1e-30).all(), (errw / (U * mass + 1e-30)).max()


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter", NORM_CASES)
def test_norm_rope_bwd(ffa, tokens, hq, hkv, d, rot, inter):
    args = norm_inputs(tokens, hq, hkv, d, rot, 7 * tokens + hq)
    grads = ffa.qk_norm_rope_bwd(*args, eps=1e-5, interleaved=inter)
    check_norm_bwd(ffa, grads, *args, 1e-5, inter)
    again = ffa.qk_norm_rope_bwd(*args, eps=1e-5, interleaved=inter)
    assert all((bits(a) == bits(b)).all() for a, b in zip(grads, again))   # a fixed order of sums


@pytest.mark.parametrize("tokens,hq,hkv,d,rot", [(12011, 7, 3, 128, 96), (9001, 11, 4, 64, 48)])
def test_norm_rope_with_several_units_a_warp(ffa, tokens, hq, hkv, d, rot):
    args = norm_inputs(tokens, hq, hkv, d, rot, tokens)
    q, k, qw, kw, t, pos = args[:6]
    pos[::7] = -1
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos, eps=1e-5)
    check_norm(qo, q, qw, t, pos, 1e-5, False)
    check_norm(ko, k, kw, t, pos, 1e-5, False)
    check_norm_bwd(ffa, ffa.qk_norm_rope_bwd(*args, eps=1e-5), *args, 1e-5, False)


def test_norm_rope_bwd_equals_differences_of_the_forward(ffa):
    """Along a random direction, against the forward's own fp64 formula at the inputs' values; the backward's dx rounds to bf16
    (2^-8 a value), so the sum's error is 2^-8 of the root of its squared terms, four times that allowed."""
    import torch
    args = norm_inputs(64, 4, 2, 128, 128, 5)
    q, k, qw, kw, t, pos, dqo, dko = args
    dq, dk, dqw, dkw = ffa.qk_norm_rope_bwd(*args)
    r = np.random.default_rng(0)
    for x, w, dout, dx, dw in ((q, qw, dqo, dq, dqw), (k, kw, dko, dk, dkw)):
        ex, ew, h = r.normal(size=x.shape), r.normal(size=w.shape), 1e-6
        f = lambda s: (S.norm_rope(f64(x) + s * h * ex, f64(w) + s * h * ew, f64(t), pos.cpu().numpy(), 1e-6, False) * f64(dout)).sum()
        num = (f(1) - f(-1)) / (2 * h)
        got = (f64(dx) * ex).sum() + (f64(dw) * ew).sum()
        slack = 4 * 2.0 ** -8 * np.sqrt(((f64(dx) * ex) ** 2).sum()) + 1e-4
        assert abs(num - got) <= slack


def test_norm_rope_padding_and_positions_behind_the_table(ffa):
    import torch
    q, k, qw, kw, t, pos, dqo, dko = norm_inputs(9, 3, 2, 64, 64, 11, max_pos=20)
    pos[2], pos[5] = -1, -2 ** 31
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos)
    check_norm(qo, q, qw, t, pos, 1e-6, False)
    assert (qo[2] == 0).all() and (ko[5] == 0).all()
    grads = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko)
    check_norm_bwd(ffa, grads, q, k, qw, kw, t, pos, dqo, dko, 1e-6, False)
    # a padded row's contents and gradients, whatever they are, reach nothing
    q2, k2, g2 = q.clone(), k.clone(), dqo.clone()
    q2[2], k2[5], g2[2] = float("nan"), float("inf"), float("nan")
    again = ffa.qk_norm_rope_bwd(q2, k2, qw, kw, t, pos, g2, dko)
    assert all((bits(a) == bits(b)).all() for a, b in zip(grads, again))
    pos[4], pos[7] = 20, 2 ** 31 - 1
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos)
    assert qo[4].isnan().all() and ko[7].isnan().all() and not qo[[0, 1, 2, 3, 5, 6, 8]].isnan().any()
    dq, dk, dqw, dkw = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko)
    assert dq[4].isnan().all() and dqw.isnan().all() and not dq[[0, 1, 2, 3, 5, 6, 8]].isnan().any()


def test_norm_rope_values_at_the_ends_of_the_range(ffa):
    import torch
    q, k, qw, kw, t, pos, _, _ = norm_inputs(8, 2, 1, 128, 128, 13)
    q, k = q.clone(), k.clone()
    q[0] = 0                      # a row of zeros: 0 / sqrt(eps)
    q[1] *= 2.0 ** -60            # all of it under eps
    q[2] *= 2.0 ** 50
    q[3, 0, 5], q[4, 1, 7] = float("nan"), float("inf")
    qo, _ = ffa.qk_norm_rope(q, k, qw, kw, t, pos)
    ok = [0, 1, 2, 5, 6, 7]
    check_norm(qo[ok], q[ok], qw, t, pos[ok], 1e-6, False)
    assert qo[3, 0].isnan().all() and not qo[3, 1].isnan().any() and qo[4, 1].isnan().any() and not qo[4, 0].isnan().any()


def test_norm_rope_no_tokens(ffa):
    import torch
    q, k, qw, kw, t, pos, dqo, dko = norm_inputs(2, 4, 2, 128, 128, 3)
    e = [x[:0] for x in (q, k, pos, dqo, dko)]
    qo, ko = ffa.qk_norm_rope(e[0], e[1], qw, kw, t, e[2])
    assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)
    ws = torch.full((ffa.qk_norm_rope_bwd_workspace_size(128),), 255, dtype=torch.uint8, device="cuda")
    _, _, dqw, dkw = ffa.qk_norm_rope_bwd(e[0], e[1], qw, kw, t, e[2], e[3], e[4], workspace=ws)
    assert (dqw == 0).all() and (dkw == 0).all()


# ---- the cache -------------------------------------------------------------------------------------------------------

def new_cache(pages, hkv, page, d, fp8):
    import torch
    c = [torch.zeros(pages, hkv, page, d, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda") for _ in "kv"]
    e = [torch.zeros(pages, hkv, page, dtype=torch.uint8, device="cuda") if fp8 else None for _ in "kv"]
    return c[0], c[1], e[0], e[1]


@pytest.mark.parametrize("tokens,hkv,d,page,fp8", [(1, 1, 64, 16, True), (1, 8, 128, 64, False), (77, 3, 128, 16, True),
                                                   (300, 2, 64, 32, True), (129, 5, 64, 128, False), (33, 32, 128, 1024, True)])
def test_cache_write_and_read(ffa, tokens, hkv, d, page, fp8):
    import torch
    g = torch.Generator().manual_seed(tokens)
    pages = tokens // page + 3
    kv = (torch.randn(tokens, 3 * hkv, d, generator=g) * torch.exp(3 * torch.randn(tokens, 3 * hkv, 1, generator=g))).bfloat16().cuda()
    k, v = kv[:, :hkv], kv[:, 2 * hkv:]   # strided views
    slots = torch.randperm(pages * page, generator=g)[:tokens].cuda()
    kc, vc, ke, ve = new_cache(pages, hkv, page, d, fp8)
    for c in (kc, vc):
        c.view(torch.uint8).fill_(0x2a)
    before = bits(kc).copy()
    ffa.kv_cache_write(k, v, kc, vc, slots, ke, ve)
    at = slots.cpu().numpy()
    for x, c, e in ((k, kc, ke), (v, vc, ve)):
        want = before.reshape(pages, hkv, page, -1).copy()
        we = np.zeros((pages, hkv, page), np.uint8)
        x64 = f64(x)
        for i in range(tokens):
            for h in range(hkv):
                if fp8:
                    want[at[i] // page, h, at[i] % page], we[at[i] // page, h, at[i] % page] = S.quantise_row(x64[i, h])
                else:
                    want[at[i] // page, h, at[i] % page] = bits(x[i, h])
        assert np.array_equal(bits(c).reshape(want.shape), want)   # every other slot untouched
        assert not fp8 or np.array_equal(e.cpu().numpy(), we)
    # read back through a page table: three sequences, one of them empty, on random pages
    order = torch.randperm(pages, generator=g)
    lens = [min(page + 3, pages * page), 0, min(2 * page - 1, max(0, (pages - 2) * page))]
    table = torch.full((3, pages), -7, dtype=torch.int32)
    used = 0
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = order[used:used + need].int()
        used += need
    if used > pages:
        lens, used = [min(page, pages * page), 0, 0], 1
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    total = sum(lens) + 5
    outs = [torch.full((total, hkv, d), 3.25, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    rk, rv = ffa.kv_cache_read(kc, vc, table.cuda(), cu, total, k=outs[0], v=outs[1], k_exp=ke, v_exp=ve)
    for out, c, e in ((rk, kc, ke), (rv, vc, ve)):
        vals = S.stored_values(bits(c).reshape(pages, hkv, page, d), e.cpu().numpy()) if fp8 else f64(c)
        ref = np.concatenate([S.gather_rows(vals, table[b].numpy(), 0, n) for b, n in enumerate(lens)])
        got = f64(out)
        # exact down to half of bf16's smallest value, 2^-133
        assert (np.abs(got[:len(ref)] - ref) <= 2.0 ** -134).all()
        assert (got[len(ref):] == 3.25).all()   # rows behind the last sequence


def test_cache_write_edge_rows(ffa):
    """Borders of the scale, ties, zeros, the smallest and largest bf16 values, NaN and infinities."""
    import torch
    d, rows = 64, []
    r = np.random.default_rng(4)
    for top in (1.75, 1.7578125, 448.0, 450.0, 2.0 ** -126 * 448, 2.0 ** -133, 3.3895314e38, 0.0, 1.0, 2.0 ** -120):
        x = r.uniform(-1, 1, d) * top
        x[0] = top
        rows.append(x)
    rows.append(np.append(448.0, np.repeat([17.0, 19.0, 21.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10, -17.0], 9)))   # ties
    rows.append(np.full(d, -0.0))
    for bad in (np.nan, np.inf, -np.inf):
        x = r.normal(size=d)
        x[33] = bad
        rows.append(x)
    k = torch.tensor(np.stack(rows)).bfloat16().cuda()[:, None, :]
    n = len(rows)
    kc, vc, ke, ve = new_cache(2, 1, 16, d, True)
    ffa.kv_cache_write(k, k, kc, vc, torch.arange(n).cuda(), ke, ve)
    got, ge = bits(kc).reshape(32, d), ke.cpu().numpy().reshape(32)
    for i in range(n):
        codes, byte = S.quantise_row(f64(k)[i, 0])
        assert ge[i] == byte and np.array_equal(got[i], codes), i
    table, cu = torch.tensor([[0, 1]], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    rk, rv = ffa.kv_cache_read(kc, vc, table, cu, n, k_exp=ke, v_exp=ve)
    assert rk[-3:].isnan().all() and not rk[:-3].isnan().any() and (bits(rk) == bits(rv)).all()


def test_cache_slots_and_pages_outside_the_cache(ffa):
    """Slots that name no row are not written; pages that name no page read as NaN, and only there."""
    import torch
    for fp8 in (False, True):
        kc, vc, ke, ve = new_cache(3, 2, 16, 128, fp8)
        k = torch.ones(6, 2, 128, dtype=torch.bfloat16, device="cuda")
        slots = torch.tensor([-1, 48, 5, 2 ** 62, -2 ** 63, 47]).cuda()
        ffa.kv_cache_write(k, k, kc, vc, slots, ke, ve)
        live = (bits(kc).reshape(3, 2, 16, -1) != 0).any(-1)
        assert live.sum() == 4 and live[0, :, 5].all() and live[2, :, 15].all()
        table = torch.tensor([[2, 3], [-1, 0], [0, 2 ** 31 - 1]], dtype=torch.int32).cuda()
        cu = torch.tensor([0, 20, 40, 90], dtype=torch.int32).cuda()   # the last one is longer than its row of pages
        rk, rv = ffa.kv_cache_read(kc, vc, table, cu, 90, k_exp=ke, v_exp=ve)
        bad = rk.isnan().all(-1).all(-1).cpu().numpy()
        want = np.zeros(90, bool)
        want[16:20] = want[20:36] = want[56:90] = True
        assert np.array_equal(bad, want) and not rk[torch.from_numpy(~want).cuda()].isnan().any()
        assert (bits(rk) == bits(rv)).all()


# ---- one-token attention ---------------------------------------------------------------------------------------------

def decode_problem(lens, hq, hkv, d, page, fp8, seed, spread=0.5, extra_pages=2):
    import torch
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-n // page)) for n in lens]
    pages, width = sum(need) + extra_pages, max(1, max(need, default=1))
    kc, vc, ke, ve = new_cache(pages, hkv, page, d, fp8)
    n = pages * page
    k = torch.randn(n, hkv, d, generator=g).bfloat16().cuda()
    v = (torch.randn(n, hkv, d, generator=g) * torch.exp(spread * torch.randn(n, hkv, 1, generator=g))).bfloat16().cuda()
    ffa_write(k, v, kc, vc, ke, ve)
    order, table, used = torch.randperm(pages, generator=g).int(), torch.full((len(lens), width), -1, dtype=torch.int32), 0
    for b, c in enumerate(need):
        table[b, :c] = order[used:used + c]
        used += c
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16().cuda()
    return dict(q=q, k_cache=kc, v_cache=vc, page_table=table.cuda(), kv_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                k_exp=ke, v_exp=ve)


def ffa_write(k, v, kc, vc, ke, ve):
    import torch
    import flexible_mask_flashattention_gb300 as m
    m.kv_cache_write(k, v, kc, vc, torch.arange(k.shape[0], device="cuda"), ke, ve)


def cache_values(p):
    pages, hkv, page, d = p["k_cache"].shape
    if p["k_exp"] is None:
        return f64(p["k_cache"]), f64(p["v_cache"])
    return tuple(S.stored_values(bits(p[n + "_cache"]).reshape(pages, hkv, page, d), p[n + "_exp"].cpu().numpy()) for n in "kv")


def check_decode(out, lse, p, scale, starts=None, sink=None, skip=()):
    kv, vv = cache_values(p)
    fp8, d = p["k_exp"] is not None, p["q"].shape[-1]
    q, lens, table, got, gl = f64(p["q"]), p["kv_lens"].cpu().numpy(), p["page_table"].cpu().numpy(), f64(out), f64(lse)
    sk = None if sink is None else f64(sink)
    for b in range(len(lens)):
        if b in skip:
            continue
        hi = max(0, int(lens[b]))
        lo = 0 if starts is None else min(max(0, int(starts[b])), hi)
        vb = S.gather_rows(vv, table[b], lo, hi)
        ro, rl, mass, size = S.decode(q[b], S.gather_rows(kv, table[b], lo, hi), vb, scale, sk)
        delta = (d + 16) * U * size
        w = (2.0 ** -11 if fp8 else 2.0 ** -16) + 2 * delta + ((hi - lo) / 16 + 32) * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ro) + w[:, None] * mass + 1e-30
        if fp8:
            tol = tol + (hi - lo) * 2.0 ** -34 * np.abs(vb).max(initial=0.0)
        err = np.abs(got[b] - ro)
        assert (err <= tol).all(), (b, hi, lo, (err / tol).max())
        fin = np.isfinite(rl)
        assert np.array_equal(gl[:, b][~fin], rl[~fin]), b
        el = np.abs(gl[:, b][fin] - rl[fin])
        assert (el <= delta[fin] + 2.0 ** -20 + 4 * U * np.abs(rl[fin])).all(), (b, el.max())


DECODE = [([1], 1, 1, 64, 16), ([777], 16, 4, 128, 16), ([0, 1, 15, 16, 17, 127, 128, 129, 255, 300], 6, 2, 128, 16),
          ([500, 3, 0, 0, 1000], 8, 1, 64, 64), ([64] * 40, 3, 3, 128, 32), ([130, 2000], 32, 2, 128, 128),
          ([901, 33], 40, 2, 64, 32), ([5000], 4, 4, 64, 1024), ([-5, 40, 2], 5, 5, 128, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d,page", DECODE)
def test_decode(ffa, lens, hq, hkv, d, page, fp8):
    import torch
    p = decode_problem(lens, hq, hkv, d, page, fp8, len(lens) + hq)
    scale = d ** -0.5
    ws = torch.full((ffa.fwd_decode_workspace_size(hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    out, lse = ffa.fwd_decode(**p, scale=scale, workspace=ws)
    check_decode(out, lse, p, scale)
    again, la = ffa.fwd_decode(**p, scale=scale)
    assert (bits(again) == bits(out)).all() and (bits(la) == bits(lse)).all()   # nothing depends on timing or on the workspace


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_window_and_sink(ffa, fp8):
    import torch
    lens = [400, 17, 16, 1, 0, 333, 64]
    starts = [100, 17, 15, -3, 5, 332, 2 ** 31 - 1]
    p = decode_problem(lens, 10, 2, 128, 32, fp8, 77)
    p["page_table"][0, :3] = -1            # pages in front of the window need not be there
    st, sink = torch.tensor(starts, dtype=torch.int32).cuda(), torch.linspace(-3, 12, 10).cuda()
    for sk in (None, sink):
        out, lse = ffa.fwd_decode(**p, scale=0.1, kv_starts=st, sink=sk)
        check_decode(out, lse, p, 0.1, starts, sk)
    sink[3] = -float("inf")
    out, lse = ffa.fwd_decode(**p, scale=0.1, kv_starts=st, sink=sink)
    check_decode(out, lse, p, 0.1, starts, sink)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_small_and_many_heads(ffa, fp8):
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 90, 700)]
    p = decode_problem(lens, 2, 1, 64, 16, fp8, 6)
    check_decode(*ffa.fwd_decode(**p, scale=0.125), p, 0.125)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_sharp_and_extreme_scores(ffa, fp8):
    """Large scores of both signs, a maximum that rises key by key, a row that is all one value, a negative scale."""
    import torch
    p = decode_problem([900, 900, 31], 8, 2, 128, 16, fp8, 21, spread=2.0)
    for scale in (3.0, -2.0, 0.0):
        check_decode(*ffa.fwd_decode(**p, scale=scale), p, scale)
    n, page = 900, 16
    k = torch.zeros(57 * page, 1, 64, dtype=torch.bfloat16)
    k[:, 0, 0] = torch.arange(57 * page).float() / 4          # scores rise with the key
    v = torch.randn(57 * page, 1, 64).bfloat16()
    kc, vc, ke, ve = new_cache(57, 1, page, 64, fp8)
    ffa_write(k.cuda(), v.cuda(), kc, vc, ke, ve)
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    q[0, :, 0], q[1, :, 0] = 4.0, -4.0
    table = torch.arange(57, dtype=torch.int32).repeat(2, 1)
    p = dict(q=q.cuda(), k_cache=kc, v_cache=vc, page_table=table.cuda(), kv_lens=torch.tensor([n, n], dtype=torch.int32).cuda(),
             k_exp=ke, v_exp=ve)
    check_decode(*ffa.fwd_decode(**p, scale=1.0), p, 1.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_values_of_very_different_sizes(ffa, fp8):
    """Rows of the cache from 2^-60 to 2^60, queries from 2^-30 to 2^30 (their scores stay small)."""
    import torch
    r = np.random.default_rng(9)
    n, d = 200, 64
    mag = 2.0 ** r.integers(-60, 61, (n, 1, 1))
    v = torch.tensor(r.normal(size=(n, 1, d)) * mag).bfloat16()
    k = torch.tensor(r.normal(size=(n, 1, d)) * 2.0 ** -12).bfloat16()
    kc, vc, ke, ve = new_cache(13, 1, 16, d, fp8)
    ffa_write(k.cuda(), v.cuda(), kc, vc, ke, ve)
    q = torch.tensor(r.normal(size=(1, 3, d)) * np.array([2.0 ** -30, 1.0, 2.0 ** 9])[None, :, None]).bfloat16()
    p = dict(q=q.cuda(), k_cache=kc, v_cache=vc, page_table=torch.arange(13, dtype=torch.int32).cuda()[None],
             kv_lens=torch.tensor([n], dtype=torch.int32).cuda(), k_exp=ke, v_exp=ve)
    check_decode(*ffa.fwd_decode(**p, scale=0.125), p, 0.125)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_reads_nothing_outside_its_range(ffa, fp8):
    """NaN in every row of the cache outside the ranges changes nothing."""
    import torch
    lens, starts = [50, 33, 100], [7, 0, 63]
    p = decode_problem(lens, 4, 2, 64, 32, fp8, 31)
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    out, lse = ffa.fwd_decode(**p, scale=0.2, kv_starts=st)
    pages, hkv, page, d = p["k_cache"].shape
    keep = np.zeros((pages, page), bool)
    for b in range(3):
        for j in range(starts[b], lens[b]):
            keep[int(p["page_table"][b, j // page]), j % page] = True
    m = torch.from_numpy(~keep).cuda()[:, None, :, None].expand(pages, hkv, page, d)
    for c in (p["k_cache"], p["v_cache"]):
        raw = c.view(torch.uint8) if fp8 else c
        raw[m] = 0x7f if fp8 else float("nan")
    o2, l2 = ffa.fwd_decode(**p, scale=0.2, kv_starts=st)
    assert (bits(out) == bits(o2)).all() and (bits(lse) == bits(l2)).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_bad_pages_and_lengths(ffa, fp8):
    import torch
    p = decode_problem([100, 100, 100, 100, 100], 4, 2, 128, 16, fp8, 41)
    good, gl = ffa.fwd_decode(**p, scale=0.1)
    p["page_table"][1, 6] = -1
    p["page_table"][2, 0] = p["k_cache"].shape[0]
    p["page_table"][3, 3] = 2 ** 31 - 1
    p["kv_lens"][4] = 7 * 16 + 1               # one key more than its pages hold
    out, lse = ffa.fwd_decode(**p, scale=0.1)
    assert (bits(out[0]) == bits(good[0])).all() and (bits(lse[:, 0]) == bits(gl[:, 0])).all()
    assert out[1:].isnan().all() and lse[:, 1:].isnan().all()
    sink = torch.zeros(4, device="cuda")
    out, lse = ffa.fwd_decode(**p, scale=0.1, sink=sink)
    assert out[1:].isnan().all() and lse[:, 1:].isnan().all() and not out[0].isnan().any()
    p["kv_lens"][4] = 2 ** 31 - 1
    assert ffa.fwd_decode(**p, scale=0.1)[0][4].isnan().all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_nan_and_infinite_inputs(ffa, fp8):
    """A NaN in a key or in the query makes that row's heads NaN, and no others."""
    import torch
    p = decode_problem([60, 60], 4, 2, 64, 16, fp8, 51)
    page, row = int(p["page_table"][0, 1]), 5
    p["k_cache"].view(torch.uint8)[page, 0, row].fill_(0x7f if fp8 else 0xff)
    p["q"][1, 3, 9] = float("nan")
    out, lse = ffa.fwd_decode(**p, scale=0.1)
    bad = out.isnan().all(-1).cpu().numpy()
    assert np.array_equal(bad, [[True, True, False, False], [False, False, False, True]])
    assert np.array_equal(lse.t().isnan().cpu().numpy(), bad) and out.isnan().any(-1).cpu().numpy().sum() == bad.sum()


def test_decode_rows_past_32_bits(ffa):
    """Pages whose rows lie more than 2^32 bytes (and 2^31 values) into the cache."""
    import torch
    page, hkv, d = 64, 4, 128
    pages = (1 << 31) // (page * hkv * d) + 40
    kc = torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(1)
    n = 150
    k, v = (torch.randn(n, hkv, d, generator=g).bfloat16().cuda() for _ in "kv")
    ids = [pages - 1, pages - 17, pages - 2]
    slots = torch.tensor([ids[j // page] * page + j % page for j in range(n)]).cuda()
    ffa.kv_cache_write(k, v, kc, vc, slots)
    table = torch.tensor([ids], dtype=torch.int32).cuda()
    q = torch.randn(1, 8, d, generator=g).bfloat16().cuda()
    rk, rv = ffa.kv_cache_read(kc, vc, table, torch.tensor([0, n], dtype=torch.int32).cuda(), n)
    assert (bits(rk) == bits(k)).all() and (bits(rv) == bits(v)).all()
    out, lse = ffa.fwd_decode(q, kc, vc, table, torch.tensor([n], dtype=torch.int32).cuda(), 0.1)
    small = dict(q=q, k_cache=k.new_zeros(3, hkv, page, d), v_cache=k.new_zeros(3, hkv, page, d), k_exp=None, v_exp=None,
                 page_table=torch.arange(3, dtype=torch.int32).cuda()[None], kv_lens=torch.tensor([n], dtype=torch.int32).cuda())
    ffa.kv_cache_write(k, v, small["k_cache"], small["v_cache"], torch.arange(n).cuda())
    check_decode(out, lse, small, 0.1)


# ---- together --------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_then_steps_equal_the_causal_forward(ffa, fp8):
    """Norm and rotation, cache write, then new tokens one at a time: each step's row against ffa.fwd over the whole
    sequence, computed from the same (for e4m3: the read-back) keys and values.  Both sides round a weight to bf16 or better
    and the output to bf16: 2 (2^-8 |out| + 2^-8 sum p|v|) covers them, with sum p|v| <= max|v|."""
    import torch
    S_, steps, hq, hkv, d, page = 200, 5, 8, 2, 128, 32
    q, k, qw, kw, t, _, _, _ = norm_inputs(S_, hq, hkv, d, d, 61)
    g = torch.Generator().manual_seed(62)
    v = torch.randn(S_, hkv, d, generator=g).bfloat16().cuda()
    pos = torch.arange(S_, dtype=torch.int32).cuda()
    pages = 9
    kc, vc, ke, ve = new_cache(pages, hkv, page, d, fp8)
    table = torch.randperm(pages, generator=g)[:7].int()[None].cuda()
    slots = table[0].long()[torch.arange(S_).cuda() // page] * page + torch.arange(S_).cuda() % page
    n = S_ - steps
    qn, kn = ffa.qk_norm_rope(q[:n], k[:n], qw, kw, t, pos[:n])
    ffa.kv_cache_write(kn, v[:n], kc, vc, slots[:n], ke, ve)
    rows = []
    for i in range(n, S_):
        q1, k1 = ffa.qk_norm_rope(q[i:i + 1], k[i:i + 1], qw, kw, t, pos[i:i + 1])
        ffa.kv_cache_write(k1, v[i:i + 1], kc, vc, slots[i:i + 1], ke, ve)
        rows.append((q1, *ffa.fwd_decode(q1, kc, vc, table, torch.tensor([i + 1], dtype=torch.int32).cuda(), d ** -0.5, ke, ve)))
    kr, vr = ffa.kv_cache_read(kc, vc, table, torch.tensor([0, S_], dtype=torch.int32).cuda(), S_, k_exp=ke, v_exp=ve)
    qs = torch.cat([r[0] for r in rows])
    plan = ffa.Plan([(0, steps, 0, S_, O.CAUSAL)], steps, S_)   # bottom-right: row i sees keys up to its own
    out, lse = ffa.fwd(qs, kr, vr, plan, d ** -0.5)
    plan.check_status()
    got, gl = torch.cat([r[1] for r in rows]), torch.cat([r[2] for r in rows], 1)
    tol = 2 * 2.0 ** -8 * (np.abs(f64(out)) + np.abs(f64(vr)).max())
    assert (np.abs(f64(got) - f64(out)) <= tol).all()
    assert np.abs(f64(gl) - f64(lse)).max() <= 1e-3


def test_first_keys_and_window_merge_like_the_sink_window_mask(ffa):
    """Two key ranges joined by lse_combine equal one attention over their union (2^-8 of each part's rounding and of the result's)."""
    import torch
    p = decode_problem([700, 90], 8, 2, 128, 64, True, 71)
    first = p["kv_lens"].clamp(max=64)
    starts = (p["kv_lens"] - 200).clamp(min=64).int()
    a = ffa.fwd_decode(p["q"], p["k_cache"], p["v_cache"], p["page_table"], first, 0.09, p["k_exp"], p["v_exp"])
    b = ffa.fwd_decode(**p, scale=0.09, kv_starts=starts)
    out, lse = ffa.lse_combine(*a, *b)
    kv, vv = cache_values(p)
    for i, n in enumerate((700, 90)):
        keys = [j for j in range(n) if j < 64 or j >= max(64, n - 200)]
        rows = [(int(p["page_table"][i, j // 64]), j % 64) for j in keys]
        ks, vs = (np.stack([x[pg, :, r] for pg, r in rows]) for x in (kv, vv))
        ro, rl, mass, _ = S.decode(f64(p["q"])[i], ks, vs, 0.09)
        assert (np.abs(f64(out)[i] - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -7 * mass).all()
        assert np.abs(f64(lse)[:, i] - rl).max() <= 1e-3


def test_training_step_through_norm_and_attention(ffa):
    """qk_norm_rope -> fwd -> bwd -> qk_norm_rope_bwd against the oracle's chain, with the tolerances of the attention's
    gradients."""
    import torch
    from ffa_testlib import check_grad
    S_, hq, hkv, d = 150, 4, 2, 64
    q, k, qw, kw, t, _, dout, _ = norm_inputs(S_, hq, hkv, d, 32, 81)
    v = norm_inputs(S_, hq, hkv, d, 32, 82)[1].contiguous()
    pos = torch.arange(S_, dtype=torch.int32).cuda()
    qn, kn = ffa.qk_norm_rope(q, k, qw, kw, t, pos, interleaved=True)
    plan = ffa.Plan([(0, S_, 0, S_, O.CAUSAL)], S_, S_)
    out, lse = ffa.fwd(qn, kn, v, plan, 0.125)
    dqn, dkn, dv = ffa.bwd(qn, kn, v, out, lse, dout, plan, 0.125)
    grads = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqn, dkn, interleaved=True)
    plan.check_status()
    p = pos.cpu().numpy()
    rq, rk = (S.norm_rope(f64(x), f64(w), f64(t), p, 1e-6, True) for x, w in ((q, qw), (k, kw)))
    a = [torch.from_numpy(x) for x in (rq, rk, f64(v), f64(dout))]
    rdq, rdk, _ = O.attention_backward(*a, [(0, S_, 0, S_, O.CAUSAL)], 0.125)
    for x, w, g, i in ((q, qw, rdq, 0), (k, kw, rdk, 1)):
        dx, dw, _ = S.norm_rope_grad(f64(x), f64(w), f64(t), p, g, 1e-6, True)
        check_grad(f64(grads[i]), dx, "dx")
        check_grad(f64(grads[2 + i]), dw, "dweight")


# ---- streams, graphs, refusals -----------------------------------------------------------------------------------------

def test_calls_on_another_stream_and_in_a_graph(ffa):
    """A captured step, replayed with new inputs and lengths in place, equals the eager calls; so do calls given a stream."""
    import torch
    p = decode_problem([200, 31, 90], 8, 2, 128, 32, True, 91)
    q, k, qw, kw, t, _, _, _ = norm_inputs(3, 8, 2, 128, 128, 92)
    pos, slots = (p["kv_lens"] - 1).contiguous(), torch.zeros(3, dtype=torch.int64, device="cuda")
    v = torch.randn(3, 2, 128, device="cuda").bfloat16()
    ws = torch.empty(ffa.fwd_decode_workspace_size(8, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 3, device="cuda")
    qo, ko = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        ffa.qk_norm_rope(q, k, qw, kw, t, pos, q_out=qo, k_out=ko, stream=stream)
        ffa.kv_cache_write(ko, v, p["k_cache"], p["v_cache"], slots, p["k_exp"], p["v_exp"], stream=stream)
        ffa.fwd_decode(qo, p["k_cache"], p["v_cache"], p["page_table"], p["kv_lens"], 0.09, p["k_exp"], p["v_exp"], out=out,
                       lse=lse, workspace=ws, stream=stream)

    def set_slots():
        j = p["kv_lens"].long() - 1
        slots.copy_(p["page_table"].long().gather(1, (j // 32)[:, None])[:, 0] * 32 + j % 32)
        pos.copy_(p["kv_lens"] - 1)

    set_slots()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    p["kv_lens"].copy_(torch.tensor([150, 32, 96], dtype=torch.int32))
    q.copy_(torch.randn(q.shape, device="cuda").bfloat16())
    set_slots()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    first = (bits(out).copy(), bits(lse).copy(), bits(p["k_cache"]).copy())
    out.zero_()
    step()
    assert (bits(out) == first[0]).all() and (bits(lse) == first[1]).all() and (bits(p["k_cache"]) == first[2]).all()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert (bits(out) == first[0]).all()
    out.zero_()
    torch.cuda.synchronize()
    step(side.cuda_stream)
    o2, _ = ffa.fwd_decode(qo, p["k_cache"], p["v_cache"], p["page_table"], p["kv_lens"], 0.09, p["k_exp"], p["v_exp"], stream=side)
    side.synchronize()
    assert (bits(out) == first[0]).all() and (bits(o2) == first[0]).all()


def test_inputs_freed_while_another_stream_still_reads_them(ffa):
    """A call that is given a busy stream keeps its inputs' memory from being handed out before it has run."""
    import torch
    q, k, qw, kw, t, pos, _, _ = norm_inputs(4096, 8, 2, 128, 128, 121)
    want = [bits(x) for x in ffa.qk_norm_rope(q, k, qw, kw, t, pos)]
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for given in (side, side.cuda_stream):
        q2, k2 = q.clone(), k.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(40):
                big @ big                     # some milliseconds of work in front of the call
        out = ffa.qk_norm_rope(q2, k2, qw, kw, t, pos, stream=given)
        del q2, k2
        junk = [torch.full((4096, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        junk += [torch.full((4096, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all((bits(a) == b).all() for a, b in zip(out, want)) and len(junk) == 8


def test_calls_from_several_threads_at_once(ffa):
    """Threads with a stream of their own, and two on one stream: every call's results are the ones it has alone."""
    import threading
    import torch
    probs = [decode_problem([300 + 40 * i, 17, 90 * i], 8, 2, 128, 32, i % 2 == 0, 200 + i) for i in range(4)]
    norms = [norm_inputs(257 + i, 6, 2, 64, 32, 300 + i) for i in range(4)]
    want = [(ffa.fwd_decode(**p, scale=0.09), ffa.qk_norm_rope_bwd(*a)) for p, a in zip(probs, norms)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    streams.append(streams[0])
    bad = []

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(60):
                got = (ffa.fwd_decode(**probs[i], scale=0.09), ffa.qk_norm_rope_bwd(*norms[i]))
                streams[i].synchronize()
                if not all((bits(a) == bits(b)).all() for x, y in zip(got, want[i]) for a, b in zip(x, y)):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_strided_views(ffa):
    """A page table that is a part of a wider one, queries that are a part of a projection's output, outputs given."""
    import torch
    p = decode_problem([200, 64, 130], 4, 2, 64, 32, True, 111)
    want = ffa.fwd_decode(**p, scale=0.1)
    wide = torch.full((3, p["page_table"].shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, 2:-3] = p["page_table"]
    qkv = torch.randn(3, 8, 64, device="cuda").bfloat16()
    qkv[:, 2:6] = p["q"]
    out, lse = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 3, device="cuda")
    got = ffa.fwd_decode(**{**p, "q": qkv[:, 2:6], "page_table": wide[:, 2:-3]}, scale=0.1, out=out, lse=lse)
    assert got[0] is out and (bits(out) == bits(want[0])).all() and (bits(lse) == bits(want[1])).all()
    cu = torch.tensor([0, 200, 264, 394], dtype=torch.int32, device="cuda")
    a = ffa.kv_cache_read(p["k_cache"], p["v_cache"], p["page_table"], cu, 394, k_exp=p["k_exp"], v_exp=p["v_exp"])
    b = ffa.kv_cache_read(p["k_cache"], p["v_cache"], wide[:, 2:-3], cu, 394, k_exp=p["k_exp"], v_exp=p["v_exp"])
    assert all((bits(x) == bits(y)).all() for x, y in zip(a, b))


def test_norm_rope_bwd_in_a_graph(ffa):
    import torch
    args = norm_inputs(333, 4, 2, 128, 128, 95)
    eager = ffa.qk_norm_rope_bwd(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ffa.qk_norm_rope_bwd(*args)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all((bits(a) == bits(b)).all() for a, b in zip(eager, got))


def test_binding_refusals(ffa):
    import torch
    q, k, qw, kw, t, pos, dqo, dko = norm_inputs(4, 4, 2, 64, 64, 97)
    p = decode_problem([20, 30], 4, 2, 64, 16, True, 98)
    kc, vc, ke, ve, q2 = p["k_cache"], p["v_cache"], p["k_exp"], p["v_exp"], p["q"]
    bf = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    slots, x = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    N, W, R, D = ffa.qk_norm_rope, ffa.kv_cache_write, ffa.kv_cache_read, ffa.fwd_decode
    pt, ln = p["page_table"], p["kv_lens"]
    bad = [
        lambda: N(q.float(), k, qw, kw, t, pos), lambda: N(q, k[:3], qw, kw, t, pos), lambda: N(q, k, qw.bfloat16(), kw, t, pos),
        lambda: N(q, k, qw, kw, t, pos.long()), lambda: N(q, k, qw, kw[:32], t, pos), lambda: N(q, k, qw, kw, t[:, 0], pos),
        lambda: N(q.transpose(0, 1), k, qw, kw, t, pos), lambda: N(q, k, qw, kw, t[:, :40].contiguous(), pos),
        lambda: N(q, k, qw, kw, t, pos, q_out=q.contiguous()[:2]), lambda: N(q, k.contiguous(), qw, kw, t, pos, k_out=q),
        lambda: N(q.contiguous()[..., ::2], k, qw, kw, t, pos),
        lambda: ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo.float(), dko), lambda: ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo[:2], dko),
        lambda: ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: W(x, x, kc, vc, slots), lambda: W(x, x, bf, bf.clone(), slots, ke, ve), lambda: W(x, x, kc, bf, slots, ke, ve),
        lambda: W(x, x, bf, bf.clone(), slots.int()), lambda: W(x[:, :1], x, bf, bf.clone(), slots), lambda: W(x, x[:3], bf, bf.clone(), slots),
        lambda: W(x, x, kc, vc, slots, ke[:1], ve), lambda: W(x, x, bf[:, :, :12].contiguous(), bf[:, :, :12].contiguous(), slots),
        lambda: R(kc, vc, pt, cu.long(), 50, k_exp=ke, v_exp=ve), lambda: R(kc, vc, pt[:1], cu, 50, k_exp=ke, v_exp=ve),
        lambda: R(kc, vc, pt, cu, -1, k_exp=ke, v_exp=ve), lambda: R(kc, vc, pt, cu, 50, k=x, k_exp=ke, v_exp=ve),
        lambda: D(q2[:1], kc, vc, pt, ln, 1.0, ke, ve), lambda: D(q2[:, :3], kc, vc, pt, ln, 1.0, ke, ve),
        lambda: D(q2, kc, vc, pt.long(), ln, 1.0, ke, ve), lambda: D(q2, kc, vc, pt, ln.long(), 1.0, ke, ve),
        lambda: D(q2, kc, vc, pt, ln, float("nan"), ke, ve), lambda: D(q2, kc, vc, pt, ln, 1.0, ke, ve, sink=torch.zeros(3, device="cuda")),
        lambda: D(q2, kc, vc, pt, ln, 1.0, ke, ve, kv_starts=ln[:1]), lambda: D(q2, kc, vc, pt, ln, 1.0, ke, ve, lse=torch.zeros(2, 4, device="cuda")),
        lambda: D(q2, kc, vc, pt, ln, 1.0, ke, ve, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: D(q2, kc, vc, pt.t().contiguous().t(), ln, 1.0, ke, ve),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ffa.FFAError):
            call()
            print("accepted:", i)
    torch.cuda.synchronize()
    out, _ = D(q2, kc, vc, pt, ln, 1.0, ke, ve)
    assert not out.isnan().any()
