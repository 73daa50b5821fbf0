"""The paged cache in 4 bits (e2m1 codes, e4m3 scales, exponent bytes): bit-exact writing, exact reading, and one-token attention over it against
the fp64 oracle, with the tolerance derived in serving_lib.py."""
import numpy as np
import pytest

from oracle import serving as S
from serving_lib import Cache, check_decode, problem, same_arrays
from test_gpu_serving import DECODE, bits, f64, ffa  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hkv,d,page", [(1, 1, 64, 16), (1, 8, 128, 64), (77, 3, 128, 16), (300, 2, 64, 32), (41, 16, 64, 16),
                                               (33, 32, 128, 1024), (19, 8, 128, 128)])
def test_write_and_read(ffa, tokens, hkv, d, page):
    """Codes, scales and bytes are the oracle's; every other row untouched; what is read back is what they stand for, and rows behind the
    last sequence stay as they were."""
    import torch
    g = torch.Generator().manual_seed(tokens + d)
    pages = tokens // page + 3
    kv = torch.randn(tokens, 3 * hkv, d, generator=g) * torch.exp(3 * torch.randn(tokens, 3 * hkv, 1, generator=g))
    kv = (kv * torch.exp(1.5 * torch.randn(tokens, 3 * hkv, d // 16, generator=g)).repeat_interleave(16, -1)).bfloat16().cuda()
    x = {"k": kv[:, :hkv], "v": kv[:, 2 * hkv:]}   # strided views
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 5:
        slots[3], slots[5] = -1, pages * page
    c = Cache(pages, hkv, page, d, "e2m1", fill=0x2a)
    want = c.arrays()
    ffa.kv_cache_write(x["k"], x["v"], c.k, c.v, slots.cuda(), **c.more())
    for n in "kv":
        c.expect(want, n, f64(x[n]), slots.tolist())
    same_arrays(c.arrays(), want)
    order = torch.randperm(pages, generator=g)
    lens = [min(page + 3, pages * page), 0, min(2 * page - 1, (pages - 2) * page)]
    table, used = torch.full((3, pages), -7, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = order[used:used + need].int()
        used += need
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    total = sum(lens) + 5
    outs = [torch.full((total, hkv, d), 3.25, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ffa.kv_cache_read(c.k, c.v, table.cuda(), cu, total, k=outs[0], v=outs[1], **c.more())
    for n, out in zip("kv", outs):
        vals = c.values(n)
        ref = np.concatenate([S.gather_rows(vals, table[b].numpy(), 0, n_) for b, n_ in enumerate(lens)])
        got = f64(out)
        assert (np.abs(got[:len(ref)] - ref) <= 2.0 ** -134).all()   # exact down to half of bf16's smallest value
        assert (got[len(ref):] == 3.25).all()


@pytest.mark.parametrize("hkv,d", [(8, 128), (3, 64), (16, 64)])
def test_rows_at_multiples_of_16_bytes_only(ffa, hkv, d):
    """Inputs and outputs 16 bytes into an allocation, token strides that are multiples of 8 values: the same as at round addresses."""
    import torch
    g = torch.Generator().manual_seed(hkv)
    n, page = 90, 32
    k, v = (torch.randn(n, hkv, d, generator=g).bfloat16().cuda() for _ in "kv")
    wide = torch.zeros(n, 2 * hkv * d + 8, dtype=torch.bfloat16, device="cuda")
    odd = [wide[:, 8 + i * hkv * d:8 + (i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2)]
    odd[0].copy_(k), odd[1].copy_(v)
    a, b = (Cache(4, hkv, page, d, "e2m1") for _ in range(2))
    slots = torch.randperm(4 * page, generator=g)[:n].cuda()
    ffa.kv_cache_write(k, v, a.k, a.v, slots, **a.more())
    ffa.kv_cache_write(*odd, b.k, b.v, slots, **b.more())
    same_arrays(a.arrays(), b.arrays())
    table, cu = torch.arange(4, dtype=torch.int32).cuda()[None], torch.tensor([0, 4 * page], dtype=torch.int32).cuda()
    want = ffa.kv_cache_read(a.k, a.v, table, cu, 4 * page, **a.more())
    out = [torch.empty(4 * page * hkv * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(4 * page, hkv, d) for _ in "kv"]
    ffa.kv_cache_read(a.k, a.v, table, cu, 4 * page, k=out[0], v=out[1], **a.more())
    assert all((bits(x) == bits(y)).all() for x, y in zip(out, want))


def test_every_scale_and_every_tie(ffa):
    """Groups whose scale runs over all e4m3 values beside one that sets the row's exponent; in them, every border between two codes, exactly
    and one bf16 step to either side; scales that are halfway between two."""
    import torch
    grid = S.e4m3_values()
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = []
    for code in range(1, 127):
        s = grid[code]
        t = torch.tensor(ties * s).bfloat16()
        steps = t.view(torch.int16)
        near = [t.double().numpy(), (steps + 1).view(torch.bfloat16).double().numpy(), (steps - 1).view(torch.bfloat16).double().numpy()]
        for shift in (0, 3, -40):
            for vals in near:
                row = np.zeros(64)
                row[0] = 2688.0                                       # n = 0
                row[16:24], row[24:32] = vals, -vals
                row[24] = 6.0 * s                                     # the group's scale is s
                row[32:40] = vals * 0.9375                            # another one, its scale from the values
                row[48] = (grid[code] + grid[code - 1]) / 2 * 6.0     # a scale halfway between two (where 6 times it is a bf16 value)
                rows.append(row * 2.0 ** shift)
    x = torch.tensor(np.stack(rows)).bfloat16().cuda()[:, None, :]
    n = len(rows)
    c = Cache(-(-n // 64), 1, 64, 64, "e2m1")
    want = c.arrays()
    ffa.kv_cache_write(x, x, c.k, c.v, torch.arange(n).cuda(), **c.more())
    for name in "kv":
        c.expect(want, name, f64(x), range(n))
    same_arrays(c.arrays(), want)


def test_edge_rows(ffa):
    """Borders of the exponent, zeros, the smallest and largest bf16 values, groups far below the row's largest, NaN and infinities."""
    import torch
    d, rows = 128, []
    r = np.random.default_rng(4)
    for top in (1.3125, 1.3203125, 2688.0, 2704.0, 2.0 ** -126 * 2688, 2.0 ** -126 * 2704, 2.0 ** -133, 3.3895314e38, 0.0, 1.0, 2.0 ** -120):
        x = r.uniform(-1, 1, d) * top
        x[0] = top
        x[32:48] *= 2.0 ** -9
        x[48:64] *= 2.0 ** -19      # its scale is 0 beside the largest
        x[64:80] *= 2.0 ** -300
        rows.append(x)
    rows.append(np.full(d, -0.0))
    for bad in (np.nan, np.inf, -np.inf):
        x = r.normal(size=d)
        x[33] = bad
        rows.append(x)
    k = torch.tensor(np.stack(rows)).bfloat16().cuda()[:, None, :]
    n = len(rows)
    c = Cache(2, 1, 16, d, "e2m1")
    want = c.arrays()
    ffa.kv_cache_write(k, k, c.k, c.v, torch.arange(n).cuda(), **c.more())
    for name in "kv":
        c.expect(want, name, f64(k), range(n))
    same_arrays(c.arrays(), want)
    table, cu = torch.tensor([[0, 1]], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    rk, rv = ffa.kv_cache_read(c.k, c.v, table, cu, n, **c.more())
    assert rk[-3:].isnan().all() and not rk[:-3].isnan().any() and (bits(rk) == bits(rv)).all()


def test_pages_outside_the_cache_read_as_nan(ffa):
    import torch
    c = Cache(3, 2, 16, 128, "e2m1")
    table = torch.tensor([[2, 3], [-1, 0], [0, 2 ** 31 - 1]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 20, 40, 90], dtype=torch.int32).cuda()
    rk, rv = ffa.kv_cache_read(c.k, c.v, table, cu, 90, **c.more())
    want = np.zeros(90, bool)
    want[16:20] = want[20:36] = want[56:90] = True
    assert np.array_equal(rk.isnan().all(-1).all(-1).cpu().numpy(), want) and (bits(rk) == bits(rv)).all()
    assert not rk[torch.from_numpy(~want).cuda()].isnan().any()


@pytest.mark.parametrize("lens,hq,hkv,d,page", DECODE + [([3000, 100], 12, 1, 64, 16), ([2500], 17, 1, 128, 64)])
def test_decode(ffa, lens, hq, hkv, d, page):
    import torch
    p, c = problem(lens, hq, hkv, d, page, "e2m1", len(lens) + hq)
    scale = d ** -0.5
    ws = torch.full((ffa.fwd_decode_workspace_size(hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    out, lse = ffa.fwd_decode(**p, scale=scale, workspace=ws)
    check_decode(out, lse, p, c, scale)
    again, la = ffa.fwd_decode(**p, scale=scale)
    assert (bits(again) == bits(out)).all() and (bits(la) == bits(lse)).all()


@pytest.mark.parametrize("hq,hkv,d,per", [(16, 4, 128, 5), (6, 2, 64, 4), (32, 2, 128, 4), (24, 1, 64, 3)])
def test_decode_with_several_blocks_a_cta(ffa, hq, hkv, d, per):
    """As many keys as give every CTA `per` blocks or more, in two sequences: the ring filled again, parts joined across CTAs."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    keys = per * sms * 64 * 12 // hkv
    p, c = problem([keys, keys // 7 + 5], hq, hkv, d, 64, "e2m1", 5)
    check_decode(*ffa.fwd_decode(**p, scale=0.3), p, c, 0.3)


def test_decode_window_and_sink(ffa):
    import torch
    lens, starts = [400, 17, 16, 1, 0, 333, 64], [100, 17, 15, -3, 5, 332, 2 ** 31 - 1]
    p, c = problem(lens, 10, 2, 128, 32, "e2m1", 77)
    p["page_table"][0, :3] = -1            # pages in front of the window need not be there
    st, sink = torch.tensor(starts, dtype=torch.int32).cuda(), torch.linspace(-3, 12, 10).cuda()
    for sk in (None, sink):
        out, lse = ffa.fwd_decode(**p, scale=0.1, kv_starts=st, sink=sk)
        check_decode(out, lse, p, c, 0.1, starts, sink=sk)


def test_decode_many_small(ffa):
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 90, 700)]
    p, c = problem(lens, 2, 1, 64, 16, "e2m1", 6)
    check_decode(*ffa.fwd_decode(**p, scale=0.125), p, c, 0.125)


def test_decode_sharp_scores_and_values_of_very_different_sizes(ffa):
    import torch
    p, c = problem([900, 900, 31], 8, 2, 128, 16, "e2m1", 21, spread=2.0)
    for scale in (3.0, -2.0, 0.0):
        check_decode(*ffa.fwd_decode(**p, scale=scale), p, c, scale)
    r = np.random.default_rng(9)
    n, d = 200, 64
    v = torch.tensor(r.normal(size=(n, 1, d)) * 2.0 ** r.integers(-60, 61, (n, 1, 1))).bfloat16().cuda()
    k = torch.tensor(r.normal(size=(n, 1, d)) * 2.0 ** -12).bfloat16().cuda()
    c = Cache(13, 1, 16, d, "e2m1")
    ffa.kv_cache_write(k, v, c.k, c.v, torch.arange(n).cuda(), **c.more())
    q = torch.tensor(r.normal(size=(1, 3, d)) * np.array([2.0 ** -30, 1.0, 2.0 ** 9])[None, :, None]).bfloat16()
    p = dict(q=q.cuda(), k_cache=c.k, v_cache=c.v, page_table=torch.arange(13, dtype=torch.int32).cuda()[None],
             kv_lens=torch.tensor([n], dtype=torch.int32).cuda(), **c.more())
    check_decode(*ffa.fwd_decode(**p, scale=0.125), p, c, 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["codes", "scales", "exponents"])
def test_decode_reads_nothing_outside_its_range(ffa, what, d):
    """Any codes, scales of NaN, or exponents of infinity in every row outside the ranges change nothing."""
    import torch
    lens, starts = [50, 33, 100], [7, 0, 63]
    p, c = problem(lens, 4, 2, d, 32, "e2m1", 31)
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    out, lse = ffa.fwd_decode(**p, scale=0.2, kv_starts=st)
    keep = np.zeros(c.shape[:3:2], bool)
    for b in range(3):
        for j in range(starts[b], lens[b]):
            keep[int(p["page_table"][b, j // 32]), j % 32] = True
    m = torch.from_numpy(~keep).cuda()[:, None, :].expand(c.shape[:3])
    for n in "kv":
        x, value = {"codes": (getattr(c, n), 0xff), "scales": (getattr(c, n + "_scale"), 0x7f), "exponents": (getattr(c, n + "_exp"), 0xff)}[what]
        x.view(torch.uint8)[m] = value
    o2, l2 = ffa.fwd_decode(**p, scale=0.2, kv_starts=st)
    assert (bits(out) == bits(o2)).all() and (bits(lse) == bits(l2)).all()


def test_decode_bad_pages_lengths_and_nan_rows(ffa):
    import torch
    p, c = problem([100] * 6, 4, 2, 128, 16, "e2m1", 41)
    good, gl = ffa.fwd_decode(**p, scale=0.1)
    p["page_table"][1, 6] = -1
    p["page_table"][2, 0] = c.shape[0]
    p["page_table"][3, 3] = 2 ** 31 - 1
    p["kv_lens"][4] = 7 * 16 + 1               # one key more than its pages hold
    c.k_scale.view(torch.uint8)[int(p["page_table"][5, 2]), 0, 5] = 0x7f   # a key of NaN, of one kv head
    sink = torch.zeros(4, device="cuda")
    for sk in (None, sink):
        out, lse = ffa.fwd_decode(**p, scale=0.1, sink=sk)
        if sk is None:
            assert (bits(out[0]) == bits(good[0])).all() and (bits(lse[:, 0]) == bits(gl[:, 0])).all()
        assert out[1:5].isnan().all() and lse[:, 1:5].isnan().all() and not out[0].isnan().any()
        assert out[5, :2].isnan().all() and not out[5, 2:].isnan().any()


def test_rows_past_32_bits(ffa):
    """Pages whose codes lie more than 2^32 bytes into the cache."""
    import torch
    page, hkv, d = 64, 4, 128
    pages = (1 << 32) // (page * hkv * d // 2) + 40
    c = Cache(pages, hkv, page, d, "e2m1")
    g = torch.Generator().manual_seed(1)
    n = 150
    k, v = (torch.randn(n, hkv, d, generator=g).bfloat16().cuda() for _ in "kv")
    ids = [pages - 1, pages - 17, pages - 2]
    slots = torch.tensor([ids[j // page] * page + j % page for j in range(n)]).cuda()
    ffa.kv_cache_write(k, v, c.k, c.v, slots, **c.more())
    q = torch.randn(1, 8, d, generator=g).bfloat16().cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    out, lse = ffa.fwd_decode(q, c.k, c.v, torch.tensor([ids], dtype=torch.int32).cuda(), lens, 0.1, **c.more())
    small = Cache(3, hkv, page, d, "e2m1")
    ffa.kv_cache_write(k, v, small.k, small.v, torch.arange(n).cuda(), **small.more())
    p = dict(q=q, k_cache=small.k, v_cache=small.v, page_table=torch.arange(3, dtype=torch.int32).cuda()[None], kv_lens=lens)
    check_decode(out, lse, p, small, 0.1)
    rk, rv = ffa.kv_cache_read(c.k, c.v, torch.tensor([ids], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(), n, **c.more())
    assert np.array_equal(f64(rk)[:n], S.gather_rows(small.values("k"), [0, 1, 2], 0, n))
    assert np.array_equal(f64(rv)[:n], S.gather_rows(small.values("v"), [0, 1, 2], 0, n))


def test_binding_refusals(ffa):
    import torch
    p, c = problem([20, 30], 4, 2, 64, 16, "e2m1", 98)
    x, slots = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.arange(4, device="cuda")
    m = c.more()
    bf = Cache(3, 2, 16, 64, "bf16")
    f8 = Cache(3, 2, 16, 64, "e4m3")
    bad = [
        lambda: ffa.kv_cache_write(x, x, c.k, c.v, slots), lambda: ffa.kv_cache_write(x, x, c.k, c.v, slots, **{**m, "k_scale": None}),
        lambda: ffa.kv_cache_write(x, x, c.k, c.v, slots, **{**m, "v_exp": None}),
        lambda: ffa.kv_cache_write(x, x, c.k, c.v, slots, **{**m, "v_scale": c.v_scale.view(torch.uint8)}),
        lambda: ffa.kv_cache_write(x, x, c.k, c.v, slots, **{**m, "k_scale": c.k_scale[..., :2]}),
        lambda: ffa.kv_cache_write(x, x, c.k, c.v[..., :16].contiguous(), slots, **m),
        lambda: ffa.kv_cache_write(x[..., :32].contiguous(), x[..., :32].contiguous(), c.k, c.v, slots, **m),
        lambda: ffa.kv_cache_write(x, x, bf.k, bf.v, slots, k_scale=c.k_scale, v_scale=c.v_scale),
        lambda: ffa.kv_cache_write(x, x, f8.k, f8.v, slots, **{**f8.more(), "k_scale": c.k_scale}),
        lambda: ffa.kv_cache_write(x, x, c.k.int(), c.v.int(), slots, **m),
        lambda: ffa.kv_cache_read(c.k, c.v, p["page_table"], torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda"), 50, k_exp=c.k_exp, v_exp=c.v_exp),
        lambda: ffa.fwd_decode(**{**p, "k_scale": None}, scale=1.0), lambda: ffa.fwd_decode(**{**p, "v_scale": c.v_scale.float()}, scale=1.0),
        lambda: ffa.fwd_decode(**{**p, "q": p["q"][..., :32].contiguous()}, scale=1.0),
    ]
    for call in bad:
        with pytest.raises(ffa.FFAError):
            call()
    assert not ffa.fwd_decode(**p, scale=1.0)[0].isnan().any()
