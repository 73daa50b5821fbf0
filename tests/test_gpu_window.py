"""One-token attention over first keys and a later range in one call, for every type of the cache, against the fp64 oracle (tolerance in
serving_lib.py)."""
import numpy as np
import pytest

from serving_lib import KINDS, check_decode, problem
from test_gpu_serving import bits, ffa  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32).cuda()


# (length, start, first): gaps of no, one and many strips, ranges that overlap or touch the first keys, either side empty, values out of range
RANGES = [(700, 500, 4), (700, 500, 16), (700, 501, 33), (700, 64, 63), (700, 63, 64), (700, 100, 200), (64, 40, 20), (64, 25, 20),
          (300, 299, 1), (300, 300, 5), (300, 400, 5), (300, 2 ** 31 - 1, 299), (300, 0, 5), (300, -7, 5), (300, 200, 0), (300, 200, -5),
          (300, 200, 2 ** 31 - 1), (1, 1, 1), (1, 0, 1), (0, 0, 5), (-4, 2, 5), (257, 256, 255), (130, 97, 65), (130, 128, 96)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d,page", [(10, 2, 128, 32), (6, 6, 64, 16), (24, 2, 64, 64), (16, 1, 128, 1024)])
def test_ranges(ffa, kind, hq, hkv, d, page):
    """Batches of more than 32 sequences and of fewer find their shares in different ways."""
    import torch
    for some in (RANGES, RANGES + RANGES[:12]):
        lens, starts, firsts = (list(x) for x in zip(*some))
        p, c = problem(lens, hq, hkv, d, page, kind, 7 * hq + d)
        sink = torch.linspace(-3, 6, hq).cuda()
        for sk in (None, sink):
            out, lse = ffa.fwd_decode(**p, scale=0.1, kv_starts=i32(starts), kv_firsts=i32(firsts), sink=sk)
            check_decode(out, lse, p, c, 0.1, starts, firsts, sk)


@pytest.mark.parametrize("kind", KINDS)
def test_without_first_keys_nothing_changes(ffa, kind):
    p, c = problem([400, 17, 1000, 3], 8, 2, 128, 32, kind, 3)
    st = i32([100, 3, 0, 5])
    a = ffa.fwd_decode(**p, scale=0.1, kv_starts=st)
    b = ffa.fwd_decode(**p, scale=0.1, kv_starts=st, kv_firsts=i32([0, 0, 0, 0]))
    assert all((bits(x) == bits(y)).all() for x, y in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (16, 2, 64)])
def test_long_sequences_with_gaps_in_every_share(ffa, kind, hq, hkv, d):
    """Units of many blocks, whose first keys and windows span CTAs."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 4 * sms * 400 // hkv
    lens = [n, n // 2 + 3, n - 77]
    starts, firsts = [n // 2 + 11, n // 3, n - 1000], [n // 3 + 5, 1000, n // 2]
    p, c = problem(lens, hq, hkv, d, 64, kind, 11)
    p["page_table"][0, n // 3 // 64 + 2:(n // 2 + 11) // 64 - 1] = -1   # pages that no key of either range lies in are not looked up
    out, lse = ffa.fwd_decode(**p, scale=0.2, kv_starts=i32(starts), kv_firsts=i32(firsts))
    check_decode(out, lse, p, c, 0.2, starts, firsts)


@pytest.mark.parametrize("kind", KINDS)
def test_reads_nothing_between_the_ranges(ffa, kind):
    """NaN in every row that no key lies in changes nothing; a page that a first key lies in has to be there."""
    import torch
    lens, starts, firsts = [500, 333, 100], [407, 200, 63], [17, 40, 3]
    p, c = problem(lens, 4, 2, 64, 32, kind, 31)
    args = dict(kv_starts=i32(starts), kv_firsts=i32(firsts))
    out, lse = ffa.fwd_decode(**p, scale=0.2, **args)
    pages, hkv, page, d = c.shape
    keep, used = np.zeros((pages, page), bool), set()
    for b in range(3):
        for j in list(range(firsts[b])) + list(range(starts[b], lens[b])):
            keep[int(p["page_table"][b, j // page]), j % page] = True
            used.add((b, j // page))
    m = torch.from_numpy(~keep).cuda()[:, None, :].expand(pages, hkv, page)
    for n in "kv":
        x = getattr(c, n + "_scale") if kind == "e2m1" else getattr(c, n)
        x.view(torch.uint8)[m] = 0x7f if kind != "bf16" else 0xff
        if kind == "bf16":
            assert x[m].isnan().all()
    for b in range(3):
        for i in range(p["page_table"].shape[1]):
            if (b, i) not in used:
                p["page_table"][b, i] = -1
    o2, l2 = ffa.fwd_decode(**p, scale=0.2, **args)
    assert (bits(out) == bits(o2)).all() and (bits(lse) == bits(l2)).all()
    p["page_table"][1, 0] = -1
    o3, l3 = ffa.fwd_decode(**p, scale=0.2, **args)
    assert o3[1].isnan().all() and l3[:, 1].isnan().all() and (bits(o3[0]) == bits(out[0])).all()


@pytest.mark.parametrize("kind", KINDS)
def test_equals_two_calls_merged(ffa, kind):
    """2^-8 of each part's and of the result's rounding."""
    import torch
    from test_gpu_serving import f64
    p, c = problem([700, 390], 8, 2, 128, 64, kind, 71)
    first, starts = i32([64, 9]), i32([500, 300])
    out, lse = ffa.fwd_decode(**p, scale=0.09, kv_starts=starts, kv_firsts=first)
    a = ffa.fwd_decode(**{**p, "kv_lens": first}, scale=0.09)
    b = ffa.fwd_decode(**p, scale=0.09, kv_starts=starts)
    mo, ml = ffa.lse_combine(*a, *b)
    assert (np.abs(f64(out) - f64(mo)) <= 2.0 ** -8 * (np.abs(f64(out)) + np.abs(f64(mo)) + np.abs(f64(a[0])) + np.abs(f64(b[0])))).all()
    assert np.abs(f64(lse) - f64(ml)).max() <= 1e-3


def test_in_a_graph_on_another_stream(ffa):
    """Ranges changed in place between replays."""
    import torch
    p, c = problem([600, 90, 333], 8, 2, 128, 32, "e2m1", 91)
    starts, firsts = i32([400, 0, 100]), i32([4, 4, 64])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ffa.fwd_decode(**p, scale=0.1, kv_starts=starts, kv_firsts=firsts)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = ffa.fwd_decode(**p, scale=0.1, kv_starts=starts, kv_firsts=firsts)
        starts.copy_(i32([500, 80, 300]))
        firsts.copy_(i32([16, 1, 1]))
        graph.replay()
    side.synchronize()
    check_decode(out, lse, p, c, 0.1, [500, 80, 300], [16, 1, 1])


def test_refusals(ffa):
    p, c = problem([20, 30], 4, 2, 64, 16, "bf16", 98)
    for firsts in (i32([1]), i32([1, 2]).long(), i32([1, 2]).cpu()):
        with pytest.raises(ffa.FFAError):
            ffa.fwd_decode(**p, scale=1.0, kv_firsts=firsts)
