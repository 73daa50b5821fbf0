"""Padding among tokens with positions of several axes, with a norm and without: q, k and every gradient against the fp64 oracle, with the tolerances of
test_gpu_serving.py and test_gpu_axes.py; what padded rows hold reaches nothing, the other tokens' rows and gradients are theirs alone."""
import numpy as np
import pytest

from test_gpu_axes import check_rope, positions, rows_of, sections
from test_gpu_serving import bits, check_norm, check_norm_bwd, f64, ffa, norm_inputs  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter,axes", [(11, 3, 2, 64, 64, False, sections(8, 12, 12)), (11, 3, 2, 64, 48, True, [i % 3 for i in range(24)]),
                                                            (203, 5, 1, 128, 96, False, [i % 4 for i in range(48)]), (64, 16, 4, 128, 128, True, sections(16, 24, 24))])
def test_padded_rows_and_the_others(ffa, tokens, hq, hkv, d, rot, inter, axes, normed):
    import torch
    q, k, qw, kw, t, _, dqo, dko = norm_inputs(tokens, hq, hkv, d, rot, tokens + d, max_pos=40)
    q, k, dqo, dko = (x.clone() for x in (q, k, dqo, dko))
    w = (qw, kw) if normed else (None, None)
    n = max(axes) + 1
    pos = positions(n, tokens, 40, tokens)
    padded = list(range(2, tokens, 3))
    for i, token in enumerate(padded):
        pos[i % n, token] = (-1, -2 ** 31, -7)[i % 3]
    pos[0, 5], pos[n - 1, 5] = 2 ** 31 - 1, -1          # padding beside a position behind the table
    good = [i for i in range(tokens) if i not in padded]
    rows, at = rows_of(t, pos, axes)
    outs = ffa.qk_norm_rope(q, k, *w, t, pos, eps=1e-5, interleaved=inter, axes=axes)
    grads = ffa.qk_norm_rope_bwd(q, k, *w, t, pos, dqo, dko, eps=1e-5, interleaved=inter, axes=axes)
    for out, x, weight, dx, dout in ((outs[0], q, qw, grads[0], dqo), (outs[1], k, kw, grads[1], dko)):
        if normed:
            check_norm(out, x, weight, rows, at, 1e-5, inter)
        else:
            check_rope(out, x, rows, at, inter)
            check_rope(dx, dout, rows, at, inter, back=True)
        assert (out[padded] == 0).all() and (dx[padded] == 0).all()
    if normed:
        check_norm_bwd(ffa, grads, q, k, qw, kw, rows, at, dqo, dko, 1e-5, inter)
    # the same without the padded tokens: rows of their own, to the bit; weight gradients are of the same terms, added in another order
    fewer = [x[good].contiguous() for x in (q, k, dqo, dko)]
    less = pos[:, good].contiguous()
    alone = ffa.qk_norm_rope(*fewer[:2], *w, t, less, eps=1e-5, interleaved=inter, axes=axes)
    back = ffa.qk_norm_rope_bwd(*fewer[:2], *w, t, less, *fewer[2:], eps=1e-5, interleaved=inter, axes=axes)
    for a, b in zip((*outs, *grads[:2]), (*alone, *back[:2])):
        assert (bits(a[good]) == bits(b)).all()
    # whatever the padded rows hold
    for i, x in enumerate((q, k, dqo, dko)):
        x[padded] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
    outs2 = ffa.qk_norm_rope(q, k, *w, t, pos, eps=1e-5, interleaved=inter, axes=axes)
    again = ffa.qk_norm_rope_bwd(q, k, *w, t, pos, dqo, dko, eps=1e-5, interleaved=inter, axes=axes)
    for a, b in zip((*outs, *grads), (*outs2, *again)):
        assert (a is None and b is None) or np.array_equal(bits(a), bits(b))
