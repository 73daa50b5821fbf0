"""kv_cache_append: the same bits as qk_norm_rope and kv_cache_write, for every type of the cache; against the fp64 oracle; and a serving run of
appends and attention over the cache."""
import numpy as np
import pytest

import oracle as O
from oracle import serving as S
from serving_lib import KINDS, Cache, check_decode, same_arrays
from test_gpu_serving import bits, check_norm, f64, ffa, norm_inputs, rope_table  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


def inputs(tokens, hq, hkv, d, rot, axes, seed, max_pos=500):
    import torch
    q, k, qw, kw, t, pos, _, _ = norm_inputs(tokens, hq, hkv, d, rot, seed, max_pos)
    g = torch.Generator().manual_seed(seed + 1)
    v = (torch.randn(tokens, hkv + 1, d, generator=g) * torch.exp(2 * torch.randn(tokens, hkv + 1, 1, generator=g))).bfloat16().cuda()[:, 1:]
    if axes is not None:
        pos = torch.randint(0, max_pos, (max(axes) + 1, tokens), generator=g, dtype=torch.int32).cuda()
    return q, k, v, qw, kw, t, pos


CASES = [(1, 1, 1, 64, 64, False, None, 16), (48, 64, 8, 128, 128, False, None, 64), (37, 6, 2, 64, 32, True, None, 16), (130, 5, 1, 128, 48, False, [i % 3 for i in range(24)], 32),
         (65, 9, 3, 64, 48, False, [0] * 7 + [1] * 17, 128), (257, 3, 3, 128, 16, True, None, 64), (100, 16, 4, 128, 96, False, None, 16),
         (515, 2, 7, 64, 64, False, [0] * 16 + [1] * 16, 1024), (700, 32, 32, 128, 128, True, [i % 4 for i in range(64)], 128)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter,axes,page", CASES)
def test_the_same_bits_as_two_calls(ffa, tokens, hq, hkv, d, rot, inter, axes, page, kind):
    """With norm and without; padding tokens, positions behind the table, slots outside the cache; every other row untouched."""
    import torch
    q, k, v, qw, kw, t, pos = inputs(tokens, hq, hkv, d, rot, axes, tokens + d)
    g = torch.Generator().manual_seed(tokens)
    pages = tokens // page + 3
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 20:
        slots[3], slots[11], slots[17] = -1, pages * page, 2 ** 50
        pos[..., 5], pos[..., 11], pos[..., 13] = -1, -3, 500
    slots = slots.cuda()
    for w in ((qw, kw), (None, None)):
        a, b = (Cache(pages, hkv, page, d, kind, fill=0x2a) for _ in range(2))
        qo = ffa.kv_cache_append(q, k, v, *w, t, pos, a.k, a.v, slots, eps=1e-5, interleaved=inter, axes=axes, **a.more())
        q2, k2 = ffa.qk_norm_rope(q, k, *w, t, pos, eps=1e-5, interleaved=inter, axes=axes)
        ffa.kv_cache_write(k2, v, b.k, b.v, slots, **b.more())
        assert (bits(qo) == bits(q2)).all()
        same_arrays(a.arrays(), b.arrays())


@pytest.mark.parametrize("kind", KINDS)
def test_many_units_a_warp(ffa, kind):
    import torch
    q, k, v, qw, kw, t, pos = inputs(14011, 7, 3, 128, 128, None, 5)
    slots = torch.randperm(14080, device="cuda")[:14011]
    a, b = (Cache(220, 3, 64, 128, kind) for _ in range(2))
    qo = ffa.kv_cache_append(q, k, v, qw, kw, t, pos, a.k, a.v, slots, **a.more())
    q2, k2 = ffa.qk_norm_rope(q, k, qw, kw, t, pos)
    ffa.kv_cache_write(k2, v, b.k, b.v, slots, **b.more())
    assert (bits(qo) == bits(q2)).all()
    same_arrays(a.arrays(), b.arrays())


@pytest.mark.parametrize("kind", KINDS)
def test_against_the_oracle(ffa, kind):
    """q and (bf16) keys within the norm's tolerance; values bit for bit; quantised keys the oracle's rows of the bf16 keys that the norm gives."""
    import torch
    axes = [0] * 16 + [1] * 24 + [2] * 24
    q, k, v, qw, kw, t, pos = inputs(70, 6, 2, 128, 128, axes, 9)
    rows, at = S.rows_of_axes(f64(t), pos.cpu().numpy(), axes)
    rows, at = torch.from_numpy(rows).cuda(), torch.from_numpy(at.astype(np.int32)).cuda()
    slots = torch.randperm(96)[:70].cuda()
    c = Cache(6, 2, 16, 128, kind)
    want = c.arrays()
    qo = ffa.kv_cache_append(q, k, v, qw, kw, t, pos, c.k, c.v, slots, axes=axes, **c.more())
    check_norm(qo, q, qw, rows, at, 1e-6, False)
    if kind == "bf16":
        check_norm(c.k[slots // 16, :, slots % 16], k, kw, rows, at, 1e-6, False)
    else:
        _, kn = ffa.qk_norm_rope(q, k, qw, kw, t, pos, axes=axes)
        check_norm(kn, k, kw, rows, at, 1e-6, False)
        c.expect(want, "k", f64(kn), slots.tolist())
    c.expect(want, "v", f64(v), slots.tolist())
    got = c.arrays()
    same_arrays(got, {n: x for n, x in want.items() if n[0] == "v" or kind != "bf16"})


@pytest.mark.parametrize("kind", KINDS)
def test_rows_with_nan_and_infinities(ffa, kind):
    """A NaN in q, k or v stays in its row: k's and v's are stored as the cache's type stores them."""
    import torch
    q, k, v, qw, kw, t, pos = inputs(8, 2, 2, 64, 64, None, 21)
    q, k, v = q.clone(), k.clone(), v.clone()
    q[1, 0, 3], k[2, 1, 5], v[3, 0, 7], v[4, 1, 9] = float("nan"), float("nan"), float("inf"), float("nan")
    a, b = (Cache(1, 2, 16, 64, kind) for _ in range(2))
    slots = torch.arange(8).cuda()
    qo = ffa.kv_cache_append(q, k, v, qw, kw, t, pos, a.k, a.v, slots, **a.more())
    q2, k2 = ffa.qk_norm_rope(q, k, qw, kw, t, pos)
    ffa.kv_cache_write(k2, v, b.k, b.v, slots, **b.more())
    assert (bits(qo) == bits(q2)).all() and qo[1, 0].isnan().all() and not qo[0].isnan().any()
    same_arrays(a.arrays(), b.arrays())


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_then_steps_with_first_keys_and_a_window(ffa, kind):
    """A prompt appended in one call, then tokens one at a time, each attending first keys and a window of the cache: every step's row against the
    oracle over what the cache holds, and against the prefill kernel under the same mask, over the keys and values read back.  Both round the
    output to bf16 and weights to bf16 or better: 2 (2^-8 |out| + 2^-8 max|v|)."""
    import torch
    n, steps, hq, hkv, d, page, first, window = 200, 6, 8, 2, 128, 32, 12, 50
    axes = [0] * 16 + [1] * 24 + [2] * 24
    q, k, v, qw, kw, t, pos = inputs(n, hq, hkv, d, d, axes, 61)
    pages = 9
    c = Cache(pages, hkv, page, d, kind)
    table = torch.randperm(pages)[:7].int()[None].cuda()
    at = torch.arange(n).cuda()
    slots = table[0].long()[at // page] * page + at % page
    args = lambda i, j: (q[i:j], k[i:j], v[i:j], qw, kw, t, pos[:, i:j].contiguous(), c.k, c.v, slots[i:j])  # noqa: E731
    ffa.kv_cache_append(*args(0, n - steps), axes=axes, **c.more())
    rows = []
    for i in range(n - steps, n):
        q1 = ffa.kv_cache_append(*args(i, i + 1), axes=axes, **c.more())
        p = dict(q=q1, k_cache=c.k, v_cache=c.v, page_table=table, kv_lens=torch.tensor([i + 1], dtype=torch.int32).cuda(), **c.more())
        st, fs = (torch.tensor([x], dtype=torch.int32).cuda() for x in (i + 1 - window, first))
        out, lse = ffa.fwd_decode(**p, scale=d ** -0.5, kv_starts=st, kv_firsts=fs)
        check_decode(out, lse, p, c, d ** -0.5, [i + 1 - window], [first])
        rows.append((q1, out, lse))
    kr, vr = ffa.kv_cache_read(c.k, c.v, table, torch.tensor([0, n], dtype=torch.int32).cuda(), n, **c.more())
    lo = n - steps + 1 - window
    # row i sees keys [lo + i, lo + i + window) and [0, first)
    plan = ffa.Plan([(0, steps, 0, first, O.FULL), (0, steps, lo, n, O.BI_CAUSAL)], steps, n)
    out, lse = ffa.fwd(torch.cat([r[0] for r in rows]), kr, vr, plan, d ** -0.5)
    plan.check_status()
    got, gl = torch.cat([r[1] for r in rows]), torch.cat([r[2] for r in rows], 1)
    assert (np.abs(f64(got) - f64(out)) <= 2 * 2.0 ** -8 * (np.abs(f64(out)) + np.abs(f64(vr)).max())).all()
    assert np.abs(f64(gl) - f64(lse)).max() <= 1e-3


def test_a_step_in_a_graph_and_on_another_stream(ffa):
    """A captured append and decode, replayed with new inputs, slots and lengths in place, equals the eager calls."""
    import torch
    B, hq, hkv, d, page = 3, 8, 2, 128, 32
    q, k, v, qw, kw, t, pos = inputs(B, hq, hkv, d, d, None, 5)
    caches = [Cache(20, hkv, page, d, "e2m1") for _ in range(2)]
    table = torch.arange(18, dtype=torch.int32).reshape(3, 6).cuda()
    lens = torch.tensor([100, 31, 90], dtype=torch.int32).cuda()
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    old = torch.randn(18 * page, hkv, d, device="cuda").bfloat16()
    for c in caches:
        ffa.kv_cache_write(old, old, c.k, c.v, torch.arange(18 * page, device="cuda"), **c.more())

    def place():
        j = lens.long() - 1
        slots.copy_(table.long().gather(1, (j // page)[:, None])[:, 0] * page + j % page)
        pos.copy_(j)

    def step(c, stream=None):
        q1 = ffa.kv_cache_append(q, k, v, qw, kw, t, pos, c.k, c.v, slots, stream=stream, **c.more())
        return ffa.fwd_decode(q1, c.k, c.v, table, lens, 0.09, stream=stream, **c.more())

    place()
    step(caches[0])
    step(caches[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    for length in ([101, 32, 96], [102, 33, 97]):
        lens.copy_(torch.tensor(length, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device="cuda").bfloat16())
        v.copy_(torch.randn(v.shape, device="cuda").bfloat16())
        place()
        graph.replay()
        want = step(caches[1])
        torch.cuda.synchronize()
        assert all((bits(a) == bits(b)).all() for a, b in zip(got, want))
        same_arrays(caches[0].arrays(), caches[1].arrays())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for given in (side, side.cuda_stream):
        other = step(caches[1], given)
        side.synchronize()
        assert all((bits(a) == bits(b)).all() for a, b in zip(other, want))


def test_no_tokens_and_refusals(ffa):
    import torch
    q, k, v, qw, kw, t, pos = inputs(4, 4, 2, 64, 64, None, 97)
    c = Cache(2, 2, 16, 64, "e4m3", fill=0x2a)
    slots, A = torch.arange(4, device="cuda"), ffa.kv_cache_append
    before = c.arrays()
    m = c.more()
    out = A(q[:0], k[:0], v[:0], qw, kw, t, pos[:0], c.k, c.v, slots[:0], **m)
    assert out.shape == (0, 4, 64)
    bad = [lambda: A(q.float(), k, v, qw, kw, t, pos, c.k, c.v, slots, **m), lambda: A(q, k[:3], v, qw, kw, t, pos, c.k, c.v, slots, **m),
           lambda: A(q, k, v[:, :1], qw, kw, t, pos, c.k, c.v, slots, **m), lambda: A(q, k, v, qw, None, t, pos, c.k, c.v, slots, **m),
           lambda: A(q, k, v, qw, kw, t, pos.long(), c.k, c.v, slots, **m), lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots.int(), **m),
           lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots[:3], **m), lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots),
           lambda: A(q, k, v, qw, kw, t[:, :40].contiguous(), pos, c.k, c.v, slots, **m), lambda: A(q, k, v, qw, kw, t, pos, c.k, c.k, slots, **m),
           lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots, axes=[0] * 32, **m), lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots, q_out=q, **m),
           lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots, q_out=torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda"), **m),
           lambda: A(q, k, v, qw, kw, t, pos[None], c.k, c.v, slots, axes=[1] * 32, **m), lambda: A(q, k, v, qw, kw, t, pos, c.k, c.v, slots, eps=-1.0, **m)]
    for call in bad:
        with pytest.raises(ffa.FFAError):
            call()
    torch.cuda.synchronize()
    same_arrays(c.arrays(), before)
