"""Columns from rot_dim on under the rotation alone: copied, whatever they and their neighbours hold (infinities, NaN, zeros of either sign), forward,
backward and on their way into a cache.

Tolerance of the columns that turn as in test_gpu_axes.py: 2^-8 |ref| + 8 u max|x| over the row, u = 2^-24.
"""
import numpy as np
import pytest

from oracle import serving as S
from serving_lib import KINDS, Cache, same_arrays
from test_gpu_serving import U, bits, f64, ffa, norm_inputs  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu

# d, rot, interleaved, axes
CASES = [(64, 32, False, None), (64, 16, True, None), (128, 48, False, [i % 3 for i in range(24)]), (128, 96, True, [0] * 20 + [1] * 28),
         (64, 48, False, [0] * 8 + [1] * 16), (128, 112, False, None)]


def with_specials(x, rot):
    """x [tokens, heads, d] with an infinity, a NaN or zeros of both signs in columns from rot on, other columns as they were."""
    import torch
    x = x.clone()
    tokens, heads, d = x.shape
    at = 0
    for t in range(0, tokens, 2):
        for h in range(heads):
            value = (float("inf"), float("-inf"), float("nan"), -0.0, 3.3e38)[at % 5]
            x[t, h, rot + (5 * at) % (d - rot)] = value
            if value == 0.0:
                x[t, h, rot:] = -0.0
            at += 1
    return x


def check(out, x, table, pos, axes, rot, inter, back=False):
    turned, raw = f64(out)[..., :rot], f64(x)[..., :rot]
    rows, at = (f64(table), pos.cpu().numpy()) if axes is None else S.rows_of_axes(f64(table), pos.cpu().numpy(), axes)
    ref = S.rope_grad(rows, at, raw, inter) if back else S.norm_rope(raw, None, rows, at, 0.0, inter)
    tol = 2.0 ** -8 * np.abs(ref) + 8 * U * np.abs(raw).max(-1, keepdims=True)
    assert (np.abs(turned - ref) <= tol).all()
    keep = np.isfinite(f64(x)[..., rot:])
    assert (bits(out[..., rot:]) == bits(x[..., rot:])).all(), np.isnan(f64(out)[..., rot:])[keep].sum()


@pytest.mark.parametrize("d,rot,inter,axes", CASES)
def test_forward_and_backward(ffa, d, rot, inter, axes):
    import torch
    q, k, _, _, t, pos, dqo, dko = norm_inputs(131, 5, 2, d, rot, d + rot)
    if axes is not None:
        g = torch.Generator().manual_seed(rot)
        pos = torch.randint(0, 500, (max(axes) + 1, 131), generator=g, dtype=torch.int32).cuda()
    q, k, dqo, dko = (with_specials(x, rot) for x in (q, k, dqo, dko))
    qo, ko = ffa.qk_norm_rope(q, k, None, None, t, pos, interleaved=inter, axes=axes)
    check(qo, q, t, pos, axes, rot, inter)
    check(ko, k, t, pos, axes, rot, inter)
    dq, dk, _, _ = ffa.qk_norm_rope_bwd(q, k, None, None, t, pos, dqo, dko, interleaved=inter, axes=axes)
    check(dq, dqo, t, pos, axes, rot, inter, back=True)
    check(dk, dko, t, pos, axes, rot, inter, back=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,rot,inter,axes", CASES)
def test_append(ffa, d, rot, inter, axes, kind):
    """q and bf16 keys as above; every cache the same bits as from two calls; padding and positions behind the table are still 0 and NaN."""
    import torch
    tokens, hkv, page = 131, 2, 32
    q, k, _, _, t, pos, _, dv = norm_inputs(tokens, 5, hkv, d, rot, d + rot + 1)
    if axes is not None:
        g = torch.Generator().manual_seed(rot)
        pos = torch.randint(0, 500, (max(axes) + 1, tokens), generator=g, dtype=torch.int32).cuda()
    q, k = with_specials(q, rot), with_specials(k, rot)
    slots = torch.randperm(5 * page, generator=torch.Generator().manual_seed(1))[:tokens].cuda()
    a, b = (Cache(5, hkv, page, d, kind) for _ in range(2))
    qo = ffa.kv_cache_append(q, k, dv, None, None, t, pos, a.k, a.v, slots, interleaved=inter, axes=axes, **a.more())
    check(qo, q, t, pos, axes, rot, inter)
    q2, k2 = ffa.qk_norm_rope(q, k, None, None, t, pos, interleaved=inter, axes=axes)
    ffa.kv_cache_write(k2, dv, b.k, b.v, slots, **b.more())
    assert (bits(qo) == bits(q2)).all()
    same_arrays(a.arrays(), b.arrays())
    if kind == "bf16":
        check(a.k[slots // page, :, slots % page], k, t, pos, axes, rot, inter)
    pos[..., 3], pos[..., 4] = -1, 500
    qo = ffa.kv_cache_append(q, k, dv, None, None, t, pos, a.k, a.v, slots, interleaved=inter, axes=axes, **a.more())
    assert (qo[3] == 0).all() and qo[4].isnan().all()
