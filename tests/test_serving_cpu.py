"""CPU checks of the norm-with-rotation, paged-cache and one-token attention calls: their oracle against what does not
depend on it, the cache's index arithmetic (lengths, pages and slots that are out of range among it) compiled for the
host, and every refusal of the C calls, which happen before anything is launched."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import serving as S

HERE = os.path.dirname(os.path.abspath(__file__))
OK, INVALID, UNSUPPORTED, OVERFLOW = 0, 1, 4, 5


# ---- the oracle

def table(max_pos, rot):
    ang = np.arange(max_pos)[:, None] * 100.0 ** (-np.arange(0, rot, 2) / rot)[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("rot,interleaved", [(16, False), (8, True), (4, False)])
def test_oracle_norm_rope_is_a_rotation_of_the_normalised_row(rot, interleaved):
    r = np.random.default_rng(0)
    x, w, t = r.normal(size=(5, 2, 16)), r.normal(size=16), table(9, rot)
    pos = np.array([0, 8, 3, -1, 9])
    out = S.norm_rope(x, w, t, pos, 1e-6, interleaved)
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w
    assert np.allclose(out[0], y[0])                                   # position 0: no rotation
    assert np.allclose((out[:3] ** 2).sum(-1), (y[:3] ** 2).sum(-1))   # lengths are kept
    assert np.allclose(out[:3, :, rot:], y[:3, :, rot:])
    assert (out[3] == 0).all() and np.isnan(out[4]).all()
    a = (0, 1) if interleaved else (0, rot // 2)                       # the first pair turns by the position in radians
    z, zr = y[2, 0, a[0]] + 1j * y[2, 0, a[1]], out[2, 0, a[0]] + 1j * out[2, 0, a[1]]
    assert np.allclose(zr, z * np.exp(3j))


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_norm_rope_gradient_equals_differences(interleaved):
    r = np.random.default_rng(1)
    x, w, t = r.normal(size=(3, 2, 8)), r.normal(size=8), table(6, 4)
    pos, dout = np.array([5, -1, 2]), r.normal(size=(3, 2, 8))
    f = lambda x_, w_: (S.norm_rope(x_, w_, t, pos, 1e-3, interleaved) * dout).sum()
    dx, dw, _ = S.norm_rope_grad(x, w, t, pos, dout, 1e-3, interleaved)
    for _ in range(12):
        ex, ew = r.normal(size=x.shape), r.normal(size=w.shape)
        h = 1e-6
        num = (f(x + h * ex, w + h * ew) - f(x - h * ex, w - h * ew)) / (2 * h)
        assert abs(num - (dx * ex).sum() - (dw * ew).sum()) < 1e-7


def test_oracle_e4m3_values_equal_torch():
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = S.stored_values(codes.numpy().reshape(1, -1), np.array([127]))[0]
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_oracle_quantise_row():
    import torch
    r = np.random.default_rng(2)
    for top in (448.0, 448.5, 1.75, 1.7500001, 1e-38, 3e38, 0.0, 1.0):
        row = np.append(r.uniform(-1, 1, 40) * top, [top, -top])
        codes, byte = S.quantise_row(row)
        n = byte - 127
        assert n >= -126 and np.abs(row).max() <= 448 * 2.0 ** n
        assert n == -126 or np.abs(row).max() > 448 * 2.0 ** (n - 1)
        want = torch.tensor(row / 2.0 ** n, dtype=torch.float64).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes, want)
        err = np.abs(S.stored_values(codes[None], np.array([byte]))[0] - row)   # half a step: 2^-4, or 2^-10 of the scale
        assert (err <= np.maximum(2.0 ** -4 * np.abs(row), 2.0 ** (n - 10)) * (1 + 1e-12)).all()
    for bad in (np.nan, np.inf, -np.inf):
        codes, byte = S.quantise_row([1.0, bad])
        assert (codes == 0x7f).all() and byte == 127


def test_oracle_decode_equals_the_attention_oracle():
    import torch
    import oracle as O
    r = np.random.default_rng(3)
    n, hq, hkv, d = 37, 6, 2, 8
    q, k, v = r.normal(size=(1, hq, d)), r.normal(size=(n, hkv, d)), r.normal(size=(n, hkv, d))
    sink = r.normal(size=hq)
    for sk in (None, sink):
        out, lse, mass, size = S.decode(q[0], k, v, 0.3, sk)
        t = [torch.from_numpy(a) for a in (q, k, v)]
        ro, rl = O.attention_forward(*t, [(0, 1, 0, n, O.FULL)], 0.3, sink=sk)
        assert np.allclose(out, ro[0]) and np.allclose(lse, rl[:, 0])
        assert (mass >= np.abs(out) - 1e-12).all() and (size >= 0).all()
    out, lse, _, _ = S.decode(q[0], k[:0], v[:0], 0.3)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_gather_rows_follows_the_page_table():
    v = np.arange(4 * 2 * 3 * 1).reshape(4, 2, 3, 1)
    got = S.gather_rows(v, [2, 0], 1, 5)
    assert got.shape == (4, 2, 1) and np.array_equal(got[:, 0, 0], [13, 14, 0, 1])


# ---- index arithmetic

def test_index_arithmetic_on_the_host(tmp_path):
    exe = str(tmp_path / "paged_index")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", os.path.join(HERE, "paged_index_main.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]


# ---- refusals (no GPU: a call that got past its checks would answer 6, FFA_ERR_CUDA)

@pytest.fixture(scope="module")
def lib():
    from flexible_mask_flashattention_gb300 import build
    build.build()
    import flexible_mask_flashattention_gb300 as ffa
    return ffa.load_library()


def at(i):
    """An aligned address for argument i; far apart, never read."""
    return (i + 1) << 32


NORM = dict(q=at(0), qs=512, k=at(1), ks=256, tokens=4, hq=4, hkv=2, d=128, qw=at(2), kw=at(3), eps=1e-6, table=at(4),
            max_pos=16, rot=128, inter=0, pos=at(5), qo=at(6), ko=at(7), stream=None)

NORM_BAD = [
    (dict(tokens=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=-1), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(d=64, rot=128), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(max_pos=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qw=None), INVALID), (dict(kw=None), INVALID),
    (dict(table=None), INVALID), (dict(pos=None), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
    (dict(q=at(0) + 8), INVALID), (dict(k=at(1) + 2), INVALID), (dict(qo=at(6) + 8), INVALID), (dict(pos=at(5) + 2), INVALID),
    (dict(table=at(4) + 4), INVALID), (dict(qs=504), INVALID), (dict(ks=255), INVALID), (dict(qs=516), INVALID),
    (dict(qs=-512), INVALID), (dict(hq=1 << 17, qs=1 << 24), OVERFLOW),
    (dict(qo=at(0)), INVALID), (dict(ko=at(0) + 64), INVALID), (dict(qo=at(7) + 128), INVALID), (dict(ko=at(4)), INVALID),
]


@pytest.mark.parametrize("change,code", NORM_BAD)
def test_norm_rope_refusals(lib, change, code):
    assert lib.ffa_qk_norm_rope(*{**NORM, **change}.values()) == code


def test_norm_rope_accepts_views_of_one_projection_and_no_tokens(lib):
    good = {**NORM, "q": at(0), "k": at(0) + 2 * 512, "qs": 1024, "ks": 1024}
    assert lib.ffa_qk_norm_rope(*good.values()) not in (INVALID, UNSUPPORTED, OVERFLOW, OK)   # got as far as CUDA
    assert lib.ffa_qk_norm_rope(*{**NORM, "tokens": 0, "q": None, "k": None, "pos": None, "qo": None, "ko": None}.values()) == OK


BWD = dict(list(NORM.items())[:16], dqo=at(6), dko=at(7), dq=at(8), dk=at(9), dqw=at(10), dkw=at(11), ws=at(12),
           ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [c for c in NORM_BAD if not set(c[0]) & {"qo", "ko"}] + [
    (dict(dqo=None), INVALID), (dict(dko=at(7) + 8), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dqw=None), INVALID), (dict(dkw=at(11) + 4), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(dq=at(6)), INVALID), (dict(dk=at(1)), INVALID), (dict(dqw=at(11) + 16), INVALID), (dict(ws=at(9)), INVALID)])
def test_norm_rope_bwd_refusals(lib, change, code):
    assert lib.ffa_qk_norm_rope_bwd(*{**BWD, **change}.values()) == code


def cache(**change):
    from flexible_mask_flashattention_gb300._lib import KVCacheC
    c = dict(k=at(20), v=at(21), k_exp=at(22), v_exp=at(23), num_pages=10, page_size=64, hkv=2, d=128, dtype=1)
    return KVCacheC(*{**c, **change}.values())


CACHE_BAD = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_exp=None), INVALID), (dict(v_exp=at(23) + 1), INVALID),
             (dict(k=at(20) + 4), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=-5), INVALID),
             (dict(num_pages=1 << 40), OVERFLOW), (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED),
             (dict(page_size=48), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED), (dict(hkv=0), INVALID),
             (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED)]


def write_args(c, **change):
    a = dict(k=at(0), ks=256, v=at(1), vs=512, tokens=3, slots=at(2), cache=ctypes.byref(c) if c else None, stream=None)
    return {**a, **change}.values()


def read_args(c, **change):
    a = dict(cache=ctypes.byref(c) if c else None, table=at(0), ts=4, max_pages=4, batch=2, cu=at(1), total=7, k=at(2),
             v=at(3), stream=None)
    return {**a, **change}.values()


def decode_args(c, **change):
    a = dict(q=at(0), qs=512, cache=ctypes.byref(c) if c else None, table=at(1), ts=4, max_pages=4, batch=2, hq=4,
             lens=at(2), starts=None, scale=0.1, sink=None, out=at(3), lse=at(4), ws=at(5), ws_bytes=1 << 30, stream=None)
    return {**a, **change}.values()


@pytest.mark.parametrize("change,code", CACHE_BAD)
def test_cache_description_refusals(lib, change, code):
    c = cache(**change)
    assert lib.ffa_kv_cache_write(*write_args(c)) == code
    assert lib.ffa_kv_cache_read(*read_args(c)) == code
    assert lib.ffa_fwd_decode(*decode_args(c)) == code


def test_a_null_cache_and_a_bf16_cache_without_exponents(lib):
    for call, args in ((lib.ffa_kv_cache_write, write_args), (lib.ffa_kv_cache_read, read_args), (lib.ffa_fwd_decode, decode_args)):
        assert call(*args(None)) == INVALID
        assert call(*args(cache(dtype=0, k_exp=None, v_exp=None))) not in (OK, INVALID, UNSUPPORTED, OVERFLOW)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(slots=at(2) + 4), INVALID), (dict(k=at(0) + 8), INVALID), (dict(ks=248), INVALID), (dict(vs=260), INVALID),
    (dict(tokens=1 << 40), OVERFLOW), (dict(tokens=0, k=None, v=None, slots=None), OK),
    (dict(k=at(20) + 512), INVALID), (dict(v=at(21) + 10 * 64 * 2 * 128 - 16), INVALID), (dict(slots=at(22)), INVALID)])
def test_cache_write_refusals(lib, change, code):
    assert lib.ffa_kv_cache_write(*write_args(cache(), **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(total=-1), INVALID), (dict(batch=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(ts=3), INVALID),
    (dict(table=None), INVALID), (dict(table=at(0) + 1), INVALID), (dict(cu=None), INVALID), (dict(cu=at(1) + 2), INVALID),
    (dict(k=None), INVALID), (dict(v=at(3) + 8), INVALID), (dict(total=1 << 31), OVERFLOW),
    (dict(total=0, k=None, v=None, cu=None, table=None), OK), (dict(batch=0), OK),
    (dict(k=at(3) + 16), INVALID), (dict(v=at(20)), INVALID), (dict(k=at(1) - 16), INVALID), (dict(v=at(0)), INVALID)])
def test_cache_read_refusals(lib, change, code):
    assert lib.ffa_kv_cache_read(*read_args(cache(), **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=3), INVALID), (dict(ts=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(q=at(0) + 8), INVALID),
    (dict(qs=504), INVALID), (dict(qs=516), INVALID), (dict(table=None), INVALID), (dict(table=at(1) + 2), INVALID),
    (dict(lens=None), INVALID), (dict(lens=at(2) + 2), INVALID), (dict(starts=at(9) + 1), INVALID), (dict(sink=at(9) + 2), INVALID),
    (dict(out=None), INVALID), (dict(out=at(3) + 2), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=100), INVALID), (dict(hq=1 << 17, qs=1 << 24), OVERFLOW), (dict(batch=(1 << 20) + 1), OVERFLOW),
    (dict(batch=0, q=None, lens=None, out=None, lse=None, ws=None), OK),
    (dict(scale=-3e38), INVALID),   # finite, but not in log2 units
    (dict(out=at(0)), INVALID), (dict(lse=at(2)), INVALID), (dict(ws=at(3) + 64), INVALID), (dict(out=at(21)), INVALID),
    (dict(lse=at(23)), INVALID), (dict(ws=at(1) - 4096), INVALID), (dict(sink=at(3)), INVALID), (dict(starts=at(4)), INVALID)])
def test_decode_refusals(lib, change, code):
    assert lib.ffa_fwd_decode(*decode_args(cache(), **change)) == code


def test_workspace_sizes(lib):
    import flexible_mask_flashattention_gb300 as ffa
    assert ffa.qk_norm_rope_bwd_workspace_size(96) == 0 and ffa.qk_norm_rope_bwd_workspace_size(64) > 0
    assert ffa.fwd_decode_workspace_size(4, 3, 128) == 0 and ffa.fwd_decode_workspace_size(4, 0, 128) == 0
    assert ffa.fwd_decode_workspace_size(4, 2, 96) == 0 and ffa.fwd_decode_workspace_size(4, 2, 64) > 0


def test_binding_refuses_tensors_that_are_not_on_the_gpu(lib):
    import torch
    import flexible_mask_flashattention_gb300 as ffa
    x, w, t = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(4, 64)
    pos, c = torch.zeros(2, dtype=torch.int32), torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    pt = torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: ffa.qk_norm_rope(x, x, w, w, t, pos), lambda: ffa.qk_norm_rope_bwd(x, x, w, w, t, pos, x, x),
                 lambda: ffa.kv_cache_write(x, x, c, c, pos.long()), lambda: ffa.kv_cache_read(c, c, pt, pos, 1),
                 lambda: ffa.fwd_decode(x, c, c, pt, pos, 1.0)):
        with pytest.raises(ffa.FFAError):
            call()


def test_binding_refuses_dimensions_beyond_32_bits():
    import torch
    import flexible_mask_flashattention_gb300 as ffa
    from flexible_mask_flashattention_gb300 import _lib
    big = 1 << 31
    for shape in ((2, big), (1, 2, big + 64)):
        with pytest.raises(ffa.FFAError) as e:
            _lib._dims(torch.empty(shape, device="meta"), "x", len(shape))
        assert e.value.code == OVERFLOW
    assert _lib._dims(torch.empty((big + 1, 2), device="meta"), "x", 2) == (big + 1, 2)
    assert _lib._dims(torch.empty((big,), device="meta"), "x", 1) == (big,)
