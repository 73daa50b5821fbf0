"""Further parity of the norm, the cache and the serving chain: rows whose tokens fill whole warps at both head dims, with padding slots
among them; interleaved pairs with several units a warp; and prefill plus steps with a tolerance of what each row weighs."""
import numpy as np
import pytest

import oracle as O
from oracle import serving as S
from test_gpu_serving import bits, check_norm, check_norm_bwd, f64, ffa, new_cache, norm_inputs  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,hkv,d", [(41, 16, 64), (19, 32, 64), (41, 8, 128), (19, 16, 128), (1, 16, 64)])
def test_cache_rows_that_fill_whole_warps(ffa, tokens, hkv, d, fp8):
    """Bit-exact codes and bytes; tokens with slots outside the cache leave everything as it was; reading back exact."""
    import torch
    g = torch.Generator().manual_seed(tokens * hkv + d)
    page, pages = 16, 5
    kv = (torch.randn(tokens, 2 * hkv, d, generator=g) * torch.exp(2 * torch.randn(tokens, 2 * hkv, 1, generator=g))).bfloat16().cuda()
    x = {"k": kv[:, :hkv], "v": kv[:, hkv:]}
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 1:
        slots[::5] = torch.tensor([-1, pages * page, 2 ** 40, -2 ** 60])[torch.arange(len(slots[::5])) % 4]
    cache = dict(zip(("k", "v", "ke", "ve"), new_cache(pages, hkv, page, d, fp8)))
    for n in "kv":
        cache[n].view(torch.uint8).fill_(0x31)
        if fp8:
            cache[n + "e"].fill_(120)
    before = {n: bits(cache[n]).reshape(pages, hkv, page, -1).copy() for n in "kv"}
    ffa.kv_cache_write(x["k"], x["v"], cache["k"], cache["v"], slots.cuda(), cache["ke"], cache["ve"])
    for n in "kv":
        want, we, x64 = before[n], np.full((pages, hkv, page), 120, np.uint8), f64(x[n])
        for i, s in enumerate(slots.tolist()):
            if not 0 <= s < pages * page:
                continue
            for h in range(hkv):
                if fp8:
                    want[s // page, h, s % page], we[s // page, h, s % page] = S.quantise_row(x64[i, h])
                else:
                    want[s // page, h, s % page] = bits(x[n][i, h])
        assert np.array_equal(bits(cache[n]).reshape(want.shape), want)
        assert not fp8 or np.array_equal(cache[n + "e"].cpu().numpy(), we)
    table = torch.tensor([[3, 0], [4, 1]], dtype=torch.int32).cuda()
    rk, rv = ffa.kv_cache_read(cache["k"], cache["v"], table, torch.tensor([0, 20, 52], dtype=torch.int32).cuda(), 52, k_exp=cache["ke"],
                               v_exp=cache["ve"])
    for n, out in (("k", rk), ("v", rv)):
        vals = S.stored_values(bits(cache[n]).reshape(pages, hkv, page, d), cache[n + "e"].cpu().numpy()) if fp8 else f64(cache[n])
        ref = np.concatenate([S.gather_rows(vals, t, 0, c) for t, c in (([3, 0], 20), ([4, 1], 32))])
        assert np.array_equal(f64(out), ref)


@pytest.mark.parametrize("tokens,hq,hkv,d,rot", [(12011, 7, 3, 128, 96), (9001, 11, 4, 64, 48)])
def test_interleaved_norm_rope_with_several_units_a_warp(ffa, tokens, hq, hkv, d, rot):
    args = norm_inputs(tokens, hq, hkv, d, rot, tokens + 1)
    q, k, qw, kw, t, pos = args[:6]
    pos[::7] = -1
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos, eps=1e-5, interleaved=True)
    check_norm(qo, q, qw, t, pos, 1e-5, True)
    check_norm(ko, k, kw, t, pos, 1e-5, True)
    check_norm_bwd(ffa, ffa.qk_norm_rope_bwd(*args, eps=1e-5, interleaved=True), *args, 1e-5, True)


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_against_the_causal_forward_by_what_each_row_weighs(ffa, fp8):
    """The last tokens one at a time over the cache, against ffa.fwd over the keys and values read back from it.  Both round the output to bf16
    (2^-8 each), the forward its weights to bf16 (2^-8 of mass = sum p |v|), the step its to 2^-11 + 2^-15 at most; 2^-12 of mass covers both sides'
    exponentials and fp32 sums.  lse: the scores' error (d + 16) 2^-24 size and 2^-20 for the logarithm, on both sides."""
    import torch
    n, steps, hq, hkv, d, page = 331, 6, 8, 2, 128, 32
    q, k, qw, kw, t, _, _, _ = norm_inputs(n, hq, hkv, d, d, 161)
    g = torch.Generator().manual_seed(162)
    v = torch.randn(n, hkv, d, generator=g).bfloat16().cuda()
    pos = torch.arange(n, dtype=torch.int32).cuda()
    kc, vc, ke, ve = new_cache(13, hkv, page, d, fp8)
    table = torch.randperm(13, generator=g)[:11].int()[None].cuda()
    slots = table[0].long()[pos.long() // page] * page + pos.long() % page
    qn, kn = ffa.qk_norm_rope(q, k, qw, kw, t, pos)
    ffa.kv_cache_write(kn, v, kc, vc, slots, ke, ve)
    first, scale = n - steps, d ** -0.5
    rows = [ffa.fwd_decode(qn[i:i + 1], kc, vc, table, torch.tensor([i + 1], dtype=torch.int32).cuda(), scale, ke, ve) for i in range(first, n)]
    kr, vr = ffa.kv_cache_read(kc, vc, table, torch.tensor([0, n], dtype=torch.int32).cuda(), n, k_exp=ke, v_exp=ve)
    plan = ffa.Plan([(0, steps, 0, n, O.CAUSAL)], steps, n)
    out, lse = ffa.fwd(qn[first:].contiguous(), kr, vr, plan, scale)
    plan.check_status()
    for i, (o, l) in enumerate(rows):
        keys = first + i + 1
        _, rl, mass, size = S.decode(f64(qn[first + i]), f64(kr[:keys]), f64(vr[:keys]), scale)
        a, b = f64(o[0]), f64(out[i])
        tol = 2 * 2.0 ** -8 * np.maximum(np.abs(a), np.abs(b)) + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15 + 2.0 ** -12) * mass
        assert (np.abs(a - b) <= tol).all(), (i, (np.abs(a - b) / tol).max())
        tol = 2 * ((d + 16) * 2.0 ** -24 * size + 2.0 ** -20 + 4 * 2.0 ** -24 * np.abs(rl))
        assert (np.abs(f64(l)[:, 0] - f64(lse)[:, i]) <= tol).all()


def test_new_tensors_are_filled_in_deterministic_mode(ffa):
    """torch fills what it allocates in this mode; so are the rows of a read behind the last sequence, which nothing writes."""
    import torch
    kc, vc, _, _ = new_cache(2, 2, 16, 64, False)
    args = kc, vc, torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.full((400, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")   # memory that the next tensors may get
    torch.use_deterministic_algorithms(True)
    try:
        k, v = ffa.kv_cache_read(*args, 400)
    finally:
        torch.use_deterministic_algorithms(False)
    for x in (k, v):
        assert (x[:3] == 0).all() and x[3:].isnan().all()


@pytest.mark.parametrize("hkv", [2, 8])
def test_a_slot_given_twice_leaves_the_others_as_they_should_be(ffa, hkv):
    import torch
    d, page, n = 128, 16, 60
    g = torch.Generator().manual_seed(hkv)
    x = torch.randn(n, hkv, d, generator=g).bfloat16().cuda()
    slots = torch.randperm(5 * page, generator=g)[:n].cuda()
    one, two = new_cache(5, hkv, page, d, True), new_cache(5, hkv, page, d, True)
    ffa.kv_cache_write(x, x, one[0], one[1], slots, one[2], one[3])
    again = torch.cat([slots, slots[:3], slots[:3]])
    ffa.kv_cache_write(torch.cat([x, 3 * x[7:10], -x[20:23]]), torch.cat([x, x[:6]]), two[0], two[1], again, two[2], two[3])
    twice = np.zeros((5, page), bool)
    twice[(slots[:3] // page).cpu().numpy(), (slots[:3] % page).cpu().numpy()] = True
    for a, b in zip(one, two):
        a, b = (bits(t).reshape(5, hkv, page, -1).transpose(0, 2, 1, 3) for t in (a, b))
        assert np.array_equal(a[~twice], b[~twice])
