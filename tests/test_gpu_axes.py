"""Norm and rotation with positions of several axes, and the rotation alone, forward and backward, against the fp64 oracle.

Tolerances as in test_gpu_serving.py.  The rotation alone is two fp32 products and a sum, rounded to bf16: 2^-8 |ref| + 4 u (|x_a| + |x_b|),
u = 2^-24, with |x_a|, |x_b| at most the row's largest.
"""
import numpy as np
import pytest

from oracle import serving as S
from test_gpu_serving import U, bits, check_norm, check_norm_bwd, f64, ffa, norm_inputs  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


def positions(axes, tokens, max_pos, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, max_pos, (axes, tokens), generator=g, dtype=torch.int32).cuda()


def sections(*counts):
    return [a for a, n in enumerate(counts) for _ in range(n)]


def rows_of(table, pos, axes):
    """The oracle's table and positions as tensors, for the checks that take tensors."""
    import torch
    rows, at = S.rows_of_axes(f64(table), pos.cpu().numpy(), axes)
    return torch.from_numpy(rows).cuda(), torch.from_numpy(at.astype(np.int32)).cuda()


# tokens, heads, d, rot, interleaved, axes: sections of whole chunks of 4 pairs and not, turns, one axis, four, an axis no pair goes by
CASES = [(1, 1, 1, 64, 64, False, sections(16, 8, 8)), (37, 6, 2, 64, 32, True, sections(3, 6, 7)), (130, 5, 1, 128, 48, False, [i % 3 for i in range(24)]),
         (65, 9, 3, 64, 48, True, [i % 2 for i in range(24)]), (257, 64, 8, 128, 128, True, sections(16, 24, 24)),
         (1000, 17, 17, 64, 64, False, sections(1, 2, 28, 1)), (2049, 2, 1, 128, 96, True, sections(48)), (3, 3, 3, 128, 16, False, [3, 0, 2, 3, 3, 0, 2, 2]),
         (515, 16, 4, 128, 128, False, [(7 * i * i) % 4 for i in range(64)])]


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter,axes", CASES)
def test_forward_and_backward(ffa, tokens, hq, hkv, d, rot, inter, axes):
    q, k, qw, kw, t, _, dqo, dko = norm_inputs(tokens, hq, hkv, d, rot, tokens + hq)
    pos = positions(max(axes) + 1, tokens, 500, tokens)
    rows, at = rows_of(t, pos, axes)
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos, eps=1e-5, interleaved=inter, axes=axes)
    check_norm(qo, q, qw, rows, at, 1e-5, inter)
    check_norm(ko, k, kw, rows, at, 1e-5, inter)
    grads = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, eps=1e-5, interleaved=inter, axes=axes)
    check_norm_bwd(ffa, grads, q, k, qw, kw, rows, at, dqo, dko, 1e-5, inter)
    again = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, eps=1e-5, interleaved=inter, axes=axes)
    assert all((bits(a) == bits(b)).all() for a, b in zip(grads, again))


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter,axes", CASES)
def test_axes_that_agree_are_one_axis(ffa, tokens, hq, hkv, d, rot, inter, axes):
    q, k, qw, kw, t, pos, dqo, dko = norm_inputs(tokens, hq, hkv, d, rot, tokens + hq)
    same = pos[None].repeat(max(axes) + 1, 1)
    pairs = [(ffa.qk_norm_rope(q, k, qw, kw, t, pos, interleaved=inter), ffa.qk_norm_rope(q, k, qw, kw, t, same, interleaved=inter, axes=axes)),
             (ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, interleaved=inter),
              ffa.qk_norm_rope_bwd(q, k, qw, kw, t, same, dqo, dko, interleaved=inter, axes=bytes(axes)))]
    for one, several in pairs:
        assert all((bits(a) == bits(b)).all() for a, b in zip(one, several))


def check_rope(out, x, rows, at, inter, back=False):
    ref = S.rope_grad(f64(rows), at.cpu().numpy(), f64(x), inter) if back else S.norm_rope(f64(x), None, f64(rows), at.cpu().numpy(), 0.0, inter)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    tol = 2.0 ** -8 * np.abs(ref) + 8 * U * np.abs(f64(x)).max(-1, keepdims=True)
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref) <= tol)[ok].all()


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,inter,axes", CASES + [(33, 4, 2, 128, 64, False, None), (9, 4, 2, 64, 16, True, None)])
def test_rotation_alone(ffa, tokens, hq, hkv, d, rot, inter, axes):
    """Without weights; the backward is the rotation back: <R x, g> = <x, R' g> up to both sides' rounding to bf16 (2^-8 of each term)."""
    import torch
    q, k, _, _, t, one, dqo, dko = norm_inputs(tokens, hq, hkv, d, rot, tokens + hq, scale=30.0)
    pos = one if axes is None else positions(max(axes) + 1, tokens, 500, tokens)
    rows, at = (t, one) if axes is None else rows_of(t, pos, axes)
    qo, ko = ffa.qk_norm_rope(q, k, None, None, t, pos, interleaved=inter, axes=axes)
    check_rope(qo, q, rows, at, inter)
    check_rope(ko, k, rows, at, inter)
    dq, dk, dqw, dkw = ffa.qk_norm_rope_bwd(q, k, None, None, t, pos, dqo, dko, interleaved=inter, axes=axes)
    assert dqw is None and dkw is None
    check_rope(dq, dqo, rows, at, inter, back=True)
    check_rope(dk, dko, rows, at, inter, back=True)
    for x, y, g, dx in ((q, qo, dqo, dq), (k, ko, dko, dk)):
        a, b = f64(y) * f64(g), f64(x) * f64(dx)
        assert abs(a.sum() - b.sum()) <= 2.0 ** -8 * (np.abs(a).sum() + np.abs(b).sum()) + 1e-20


def test_gradient_equals_differences(ffa):
    """Along a random direction, against the forward's own fp64 formula; dx rounds to bf16 (2^-8 a value), four times the root of its squares allowed."""
    args = norm_inputs(64, 4, 2, 128, 128, 5)
    q, k, qw, kw, t, _, dqo, dko = args
    axes = sections(16, 24, 24)
    pos = positions(3, 64, 500, 8)
    rows, at = S.rows_of_axes(f64(t), pos.cpu().numpy(), axes)
    dq, dk, dqw, dkw = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, axes=axes)
    r = np.random.default_rng(0)
    for x, w, dout, dx, dw in ((q, qw, dqo, dq, dqw), (k, kw, dko, dk, dkw)):
        ex, ew, h = r.normal(size=x.shape), r.normal(size=w.shape), 1e-6
        f = lambda s: (S.norm_rope(f64(x) + s * h * ex, f64(w) + s * h * ew, rows, at, 1e-6, False) * f64(dout)).sum()  # noqa: E731
        num = (f(1) - f(-1)) / (2 * h)
        got = (f64(dx) * ex).sum() + (f64(dw) * ew).sum()
        assert abs(num - got) <= 4 * 2.0 ** -8 * np.sqrt(((f64(dx) * ex) ** 2).sum()) + 1e-4


@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("axes", [sections(8, 12, 12), [i % 3 for i in range(32)]])
def test_padding_and_positions_behind_the_table(ffa, axes, normed):
    """A negative position on any axis is padding, even beside one behind the table; padded rows' contents reach nothing."""
    import torch
    q, k, qw, kw, t, _, dqo, dko = norm_inputs(11, 3, 2, 64, 64, 11, max_pos=20)
    w = (qw, kw) if normed else (None, None)
    pos = positions(3, 11, 20, 12)
    pos[0, 2], pos[2, 5], pos[1, 8], pos[0, 8] = -1, -2 ** 31, -7, 2 ** 31 - 1
    good = [i for i in range(11) if i not in (2, 5, 8)]
    qo, ko = ffa.qk_norm_rope(q, k, *w, t, pos, axes=axes)
    rows, at = rows_of(t, pos, axes)
    if normed:
        check_norm(qo, q, qw, rows, at, 1e-6, False)
    else:
        check_rope(qo, q, rows, at, False)
    assert (qo[[2, 5, 8]] == 0).all() and (ko[[2, 5, 8]] == 0).all()
    grads = ffa.qk_norm_rope_bwd(q, k, *w, t, pos, dqo, dko, axes=axes)
    q2, k2, g2 = q.clone(), k.clone(), dqo.clone()
    q2[2], k2[5], g2[8] = float("nan"), float("inf"), float("nan")
    again = ffa.qk_norm_rope_bwd(q2, k2, *w, t, pos, g2, dko, axes=axes)
    assert all(a is None or (bits(a) == bits(b)).all() for a, b in zip(grads, again))
    assert (grads[0][[2, 5, 8]] == 0).all() and not grads[0].isnan().any()
    pos[1, 4], pos[2, 7] = 20, 2 ** 31 - 1
    left = [i for i in range(11) if i not in (4, 7)]
    qo, ko = ffa.qk_norm_rope(q, k, *w, t, pos, axes=axes)
    assert qo[4].isnan().all() and ko[7].isnan().all() and not qo[left].isnan().any()
    dq, dk, dqw, dkw = ffa.qk_norm_rope_bwd(q, k, *w, t, pos, dqo, dko, axes=axes)
    assert dq[4].isnan().all() and dk[7].isnan().all() and not dq[left].isnan().any()
    assert not normed or (dqw.isnan().all() and dkw.isnan().all())
    assert len(good) == 8


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,axes", [(12011, 7, 3, 128, 96, sections(16, 16, 16)), (9001, 11, 4, 64, 48, [i % 3 for i in range(24)]),
                                                         (12011, 9, 3, 128, 128, sections(16, 24, 24)), (9001, 13, 5, 64, 64, [i % 4 for i in range(32)]),
                                                         (9001, 11, 4, 64, 64, sections(8, 12, 12)), (9001, 4, 1, 128, 96, [i % 3 for i in range(48)])])
def test_several_units_a_warp(ffa, tokens, hq, hkv, d, rot, axes):
    q, k, qw, kw, t, _, dqo, dko = norm_inputs(tokens, hq, hkv, d, rot, tokens)
    pos = positions(max(axes) + 1, tokens, 500, tokens)
    pos[1, ::7] = -1
    rows, at = rows_of(t, pos, axes)
    qo, ko = ffa.qk_norm_rope(q, k, qw, kw, t, pos, eps=1e-5, axes=axes)
    check_norm(qo, q, qw, rows, at, 1e-5, False)
    check_norm(ko, k, kw, rows, at, 1e-5, False)
    grads = ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, eps=1e-5, axes=axes)
    check_norm_bwd(ffa, grads, q, k, qw, kw, rows, at, dqo, dko, 1e-5, False)
    q1, k1 = ffa.qk_norm_rope(q, k, None, None, t, pos, axes=axes)
    check_rope(q1, q, rows, at, False)


def test_no_tokens(ffa):
    import torch
    q, k, qw, kw, t, _, dqo, dko = norm_inputs(2, 4, 2, 128, 128, 3)
    pos, axes = torch.zeros(3, 0, dtype=torch.int32, device="cuda"), sections(16, 24, 24)
    for w in ((qw, kw), (None, None)):
        qo, ko = ffa.qk_norm_rope(q[:0], k[:0], *w, t, pos, axes=axes)
        assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)
        grads = ffa.qk_norm_rope_bwd(q[:0], k[:0], *w, t, pos, dqo[:0], dko[:0], axes=axes)
        assert grads[0].shape == (0, 4, 128) and (grads[2] is None or (grads[2] == 0).all())


def test_in_a_graph_and_on_another_stream(ffa):
    """Positions changed in place between replays; the axes belong to the captured call."""
    import torch
    q, k, qw, kw, t, _, dqo, dko = norm_inputs(333, 4, 2, 128, 128, 95)
    axes, pos = [i % 3 for i in range(64)], positions(3, 333, 500, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        return (*ffa.qk_norm_rope(q, k, qw, kw, t, pos, axes=axes, stream=stream),
                *ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, axes=axes, stream=stream),
                *ffa.qk_norm_rope_bwd(q, k, None, None, t, pos, dqo, dko, axes=axes, stream=stream)[:2])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    pos.copy_(positions(3, 333, 500, 2))
    for _ in range(2):
        graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all((bits(a) == bits(b)).all() for a, b in zip(got, want))
    other = step(side)
    side.synchronize()
    assert all((bits(a) == bits(b)).all() for a, b in zip(other, want))


def test_refusals(ffa):
    import torch
    q, k, qw, kw, t, one, dqo, dko = norm_inputs(4, 4, 2, 64, 64, 97)
    pos, axes = positions(3, 4, 500, 1), sections(8, 12, 12)
    N = ffa.qk_norm_rope
    bad = [lambda: N(q, k, qw, kw, t, pos), lambda: N(q, k, qw, kw, t, one, axes=axes), lambda: N(q, k, qw, kw, t, pos, axes=axes[:-1]),
           lambda: N(q, k, qw, kw, t, pos, axes=axes + [0]), lambda: N(q, k, qw, kw, t, pos, axes=[3] * 32), lambda: N(q, k, qw, kw, t, pos, axes=[-1] * 32),
           lambda: N(q, k, qw, kw, t, pos, axes=[300] * 32), lambda: N(q, k, qw, kw, t, pos, axes="ab"), lambda: N(q, k, qw, kw, t, pos.long(), axes=axes),
           lambda: N(q, k, qw, kw, t, pos.t().contiguous().t(), axes=axes), lambda: N(q, k, qw, kw, t, pos[:, :3], axes=axes),
           lambda: N(q, k, qw, None, t, pos, axes=axes), lambda: N(q, k, None, kw, t, one), lambda: N(q, k, qw, kw, t, positions(5, 4, 500, 1), axes=axes),
           lambda: N(q, k, qw, kw, t, pos[:0], axes=axes), lambda: N(q, k, qw, kw, t, pos.cpu(), axes=axes),
           lambda: ffa.qk_norm_rope_bwd(q, k, None, None, t, pos, dqo[:2], dko, axes=axes),
           lambda: ffa.qk_norm_rope_bwd(q, k, qw, kw, t, pos, dqo, dko, axes=[0, 1, 2])]
    for call in bad:
        with pytest.raises(ffa.FFAError):
            call()
    assert not N(q, k, qw, kw, t, pos, axes=axes)[0].isnan().any()
