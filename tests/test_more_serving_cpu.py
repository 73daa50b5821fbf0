"""CPU checks of the 4-bit cache and of first keys beside a range: the oracle against what does not depend on it, the index arithmetic compiled
for the host, and the C calls' refusals."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import serving as S
from test_serving_cpu import BWD, INVALID, NORM, NORM_BAD, OK, OVERFLOW, UNSUPPORTED, at, cache, decode_args, lib, read_args, table, write_args  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))


def test_oracle_e2m1_values():
    """2 exponent bits with a bias of 1 and 1 mantissa bit; exponent 0 without the leading one."""
    for code in range(8):
        e, m = code >> 1, code & 1
        assert S.E2M1[code] == ((1 + m / 2) * 2.0 ** (e - 1) if e else m / 2)


def test_oracle_quantise_row4():
    r = np.random.default_rng(2)
    for top in (2688.0, 2689.0, 1.3125, 1.3126, 1e-38, 3e38, 0.0, 1.0):
        row = np.append(r.uniform(-1, 1, 46) * top, [top, -top])
        row[16:32] *= 2.0 ** -8
        codes, scales, byte = S.quantise_row4(row)
        n = byte - 127
        assert n >= -126 and np.abs(row).max() <= 2688 * 2.0 ** n
        assert n == -126 or np.abs(row).max() > 2688 * 2.0 ** (n - 1)
        vals = S.stored_values4(S.packed_codes(codes)[None], scales[None], np.array([byte]))[0]
        s = S.e4m3_values()[scales].repeat(16) * 2.0 ** n
        grid = np.concatenate([-S.E2M1[::-1], S.E2M1])
        best = np.abs(row[:, None] - grid * s[:, None]).min(1)      # no representable value is nearer
        assert (np.abs(vals - row) <= best * (1 + 1e-12)).all()
        g = np.abs(row.reshape(-1, 16)).max(1) / 6 / 2.0 ** n
        assert (np.abs(S.e4m3_values()[scales] - g) <= np.abs(S.e4m3_values()[:, None] - g).min(0) * (1 + 1e-12)).all()
    for z, code in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)):   # ties to the even code
        codes, scales, byte = S.quantise_row4(np.append([6.0 * 448], np.full(15, z * 448)))
        assert scales[0] == 126 and byte == 127 and (codes[1:] == code).all() and codes[0] == 7
    for bad in (np.nan, np.inf, -np.inf):
        codes, scales, byte = S.quantise_row4(np.append(np.zeros(31), bad))
        assert (scales == 0x7f).all() and byte == 127
        assert np.isnan(S.stored_values4(S.packed_codes(codes)[None], scales[None], np.array([byte]))).all()


def test_visible_keys():
    assert S.visible_keys(5, 3, 2) == [0, 1, 3, 4] and S.visible_keys(5, 1, 2) == list(range(5)) and S.visible_keys(3, 9, 2) == [0, 1]
    assert S.visible_keys(-1, 0, 4) == [] and S.visible_keys(4, -2, 0) == [0, 1, 2, 3]


MAIN = r"""
#include <cstdio>
#include <set>
#include <vector>
#include "%s/../flexible_mask_flashattention_gb300/csrc/paged.cuh"
using namespace ffa;
static int fails = 0;
int main() {
  for (int page_log2 : {4, 5, 7})
    for (int strip : {16, 32, 64})
      for (int warps : {8, 12})
        for (int len = -1; len <= 300; len += len < 0 ? 1 : 13)
          for (int start = -1; start <= 304; start += 7)
            for (int first : {-1, 0, 1, 4, 15, 16, 17, 31, 33, 63, 64, 65, 100, 129, 200, 299, 301, 2147483647}) {
              const int max_pages = (300 >> page_log2) + 1, block = strip * warps;
              const KeyRange r = key_range(len, start, first, max_pages, page_log2, strip);
              std::set<int64_t> want, got, pages, looked;
              for (int64_t j = 0; j < len; ++j)
                if (j < first || j >= start) want.insert(j), pages.insert(j >> page_log2);
              const int64_t n = range_blocks(r, block, strip);
              for (int64_t i = 0; i < n * warps; ++i) {
                const int64_t key = range_first(r, strip) + i * strip;   // as counted, without the gap
                if (key >= r.end) continue;
                const int64_t real = key_of<int64_t>(key, r.first, r.gap);
                for (int g = 0; g < strip; g += 16) {
                  bool some = r.end - key > g && (r.start - key < g + 16 || r.first - key > g);
                  if (some) looked.insert((real + g) >> page_log2);
                  for (int k = g; k < g + 16; ++k)
                    if (k < r.end - key && (k >= r.start - key || k < r.first - key)) {
                      if (!some) ++fails, std::printf("a key in a group without one\n");
                      if (!got.insert(real + k).second) ++fails, std::printf("a key twice\n");
                    }
                }
              }
              if (want != got) ++fails, std::printf("len %%d start %%d first %%d strip %%d page %%d: other keys (%%zu, %%zu)\n", len, start, first, strip, page_log2, want.size(), got.size());
              if (pages != looked) ++fails, std::printf("len %%d start %%d first %%d strip %%d page %%d: other pages\n", len, start, first, strip, page_log2);
              if (first <= 0) {
                const KeyRange o = key_range(len, start, max_pages, page_log2);
                if (o.start != r.start || o.end != r.end || o.bad != r.bad || r.first || r.gap) ++fails, std::printf("without first keys: another range\n");
              }
              if (fails > 20) return 1;
            }
  const KeyRange far = key_range(2147483647, 2147483000, 1000000000, int64_t{1} << 27, 4, 64);
  if (far.gap <= 0 || far.start < 0 || far.end < 0 || key_of<int64_t>(far.start / 64 * 64, far.first, far.gap) != 2147483000 / 64 * 64) ++fails, std::printf("far\n");
  if (!key_range(161, 100, 5, 10, 4, 16).bad || key_range(160, 100, 5, 10, 4, 16).bad) ++fails, std::printf("bad lengths\n");
  // 2 chunks a row (4 bits, d = 64): a permutation; each way of reading touches every bank once a pass
  std::set<int> all;
  for (int key = 0; key < 16; ++key)
    for (int c = 0; c < 2; ++c) all.insert(strip_chunk(key, c, 2));
  if (all.size() != 32 || *all.begin() != 0 || *all.rbegin() != 31) ++fails, std::printf("cpr 2\n");
  for (int base : {0, 8})
    for (int half = 0; half < 2; ++half) {   // K: 8 bytes a lane, 16 lanes a pass: rows 4 half .. 4 half + 3
      std::set<int> banks;
      for (int k = 0; k < 4; ++k)
        for (int t = 0; t < 4; ++t) banks.insert((strip_chunk(base + 4 * half + k, t >> 1, 2) * 4 + 2 * (t & 1)) %% 32);
      if (banks.size() != 16) ++fails, std::printf("K, cpr 2\n");
    }
  for (int o = 0; o < 4; ++o) {              // V: 4 bytes a lane, keys 2t + (o & 1) + 8 (o >> 1)
    std::set<int> banks;
    for (int t = 0; t < 4; ++t)
      for (int n = 0; n < 8; ++n) banks.insert((strip_chunk(2 * t + (o & 1) + 8 * (o >> 1), n >> 2, 2) * 4 + (n & 3)) %% 32);
    if (banks.size() != 32) ++fails, std::printf("V, cpr 2\n");
  }
  std::printf("%%d failures\n", fails);
  return fails != 0;
}
"""


def test_index_arithmetic_with_first_keys(tmp_path):
    src, exe = tmp_path / "ranges.cpp", str(tmp_path / "ranges")
    src.write_text(MAIN % HERE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-1500:]


def cache4(**change):
    from flexible_mask_flashattention_gb300._lib import KVCacheC
    c = dict(k=at(20), v=at(21), k_exp=at(22), v_exp=at(23), num_pages=10, page_size=64, hkv=2, d=128, dtype=4, k_scale=at(24), v_scale=at(25))
    return KVCacheC(*{**c, **change}.values())


@pytest.mark.parametrize("change", [dict(k_scale=None), dict(v_scale=None), dict(k_scale=at(24) + 8), dict(v_scale=at(25) + 1), dict(k_exp=None),
                                    dict(v_exp=None), dict(v_exp=at(23) + 4)])
def test_cache_in_4_bits_refusals(lib, change):  # noqa: F811
    c = cache4(**change)
    for call, args in ((lib.ffa_kv_cache_write, write_args), (lib.ffa_kv_cache_read, read_args), (lib.ffa_fwd_decode, decode_args)):
        assert call(*args(c)) == INVALID


def test_cache_in_4_bits_is_taken_and_its_arrays_overlap_nothing(lib):  # noqa: F811
    c = cache4()
    good = (OK, INVALID, UNSUPPORTED, OVERFLOW)
    for call, args in ((lib.ffa_kv_cache_write, write_args), (lib.ffa_kv_cache_read, read_args), (lib.ffa_fwd_decode, decode_args)):
        assert call(*args(c)) not in good   # got as far as CUDA
    end = 10 * 64 * 2 * 8                   # bytes of the scales
    assert lib.ffa_kv_cache_write(*write_args(c, slots=at(24) + end - 8)) == INVALID
    assert lib.ffa_kv_cache_write(*write_args(c, k=at(25))) == INVALID
    assert lib.ffa_kv_cache_write(*write_args(c, v=at(20) + 10 * 64 * 2 * 64 - 16)) == INVALID
    assert lib.ffa_kv_cache_write(*write_args(c, v=at(20) + 10 * 64 * 2 * 64)) not in good   # behind the codes
    assert lib.ffa_kv_cache_read(*read_args(c, v=at(24) + end - 16)) == INVALID
    assert lib.ffa_fwd_decode(*decode_args(c, out=at(25))) == INVALID


def window_args(c, **change):
    a = dict(q=at(0), qs=512, cache=ctypes.byref(c), table=at(1), ts=4, max_pages=4, batch=2, hq=4, lens=at(2), starts=None,
             firsts=at(9), scale=0.1, sink=None, out=at(3), lse=at(4), ws=at(5), ws_bytes=1 << 30, stream=None)
    return {**a, **change}.values()


@pytest.mark.parametrize("change,code", [(dict(firsts=at(9) + 2), INVALID), (dict(out=at(9)), INVALID), (dict(firsts=at(4) + 16), INVALID),
                                         (dict(scale=float("nan")), INVALID), (dict(batch=0, firsts=None), OK), (dict(hq=3), INVALID)])
def test_decode_window_refusals(lib, change, code):  # noqa: F811
    assert lib.ffa_fwd_decode_window(*window_args(cache(), **change)) == code


def test_decode_window_is_taken(lib):  # noqa: F811
    for c in (cache(), cache4(), cache(dtype=0, k_exp=None, v_exp=None)):
        for firsts in (None, at(9)):
            assert lib.ffa_fwd_decode_window(*window_args(c, firsts=firsts)) not in (OK, INVALID, UNSUPPORTED, OVERFLOW)


# ---- positions of several axes, the rotation alone, and the append

def test_oracle_rows_of_axes():
    t, r = table(9, 16), np.random.default_rng(0)
    pos = np.array([[0, 8, -1, 9, 3], [5, 2, 4, 4, 3], [1, 1, 1, -7, 3]])
    axes = [0, 0, 1, 2, 1, 0, 2, 2]
    rows, at_ = S.rows_of_axes(t, pos, axes)
    x = r.normal(size=(5, 2, 16))
    out = S.norm_rope(x, None, rows, at_, 0.0, False)
    assert (out[2] == 0).all() and (out[3] == 0).all()          # padding, even beside a position behind the table
    for i in (0, 1, 4):
        for pair in range(8):
            z = (x[i, :, pair] + 1j * x[i, :, pair + 8]) * np.exp(1j * pos[axes[pair], i] * 100.0 ** (-2 * pair / 16))
            assert np.allclose(out[i, :, pair], z.real) and np.allclose(out[i, :, pair + 8], z.imag)
    pos[2, 3] = 0
    assert np.isnan(S.norm_rope(x, None, *S.rows_of_axes(t, pos, axes), 0.0, False)[3]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rope_grad_is_the_transpose(interleaved):
    r = np.random.default_rng(1)
    x, g, t, pos = r.normal(size=(4, 3, 8)), r.normal(size=(4, 3, 8)), table(6, 4), np.array([5, -1, 2, 0])
    assert np.isclose((S.norm_rope(x, None, t, pos, 0.0, interleaved) * g).sum(), (x * S.rope_grad(t, pos, g, interleaved)).sum())


PAIRS = (ctypes.c_uint8 * 64)(*([0] * 16 + [1] * 24 + [2] * 24))
BAD_PAIRS = (ctypes.c_uint8 * 64)(*([0] * 63 + [3]))
AXES = dict(list(NORM.items())[:16], n=3, pairs=ctypes.cast(PAIRS, ctypes.c_void_p), qo=at(6), ko=at(7), stream=None)
AXES_BWD = dict(list(BWD.items())[:16], n=3, pairs=ctypes.cast(PAIRS, ctypes.c_void_p), **dict(list(BWD.items())[16:]))
AXES_BAD = [(dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(n=5), UNSUPPORTED), (dict(n=2), INVALID), (dict(pairs=None), INVALID),
            (dict(pairs=ctypes.cast(BAD_PAIRS, ctypes.c_void_p)), INVALID), (dict(qw=None), INVALID), (dict(kw=None), INVALID)]


@pytest.mark.parametrize("change,code", [c for c in NORM_BAD if not set(c[0]) & {"hq"}] + AXES_BAD)
def test_norm_rope_axes_refusals(lib, change, code):  # noqa: F811
    assert lib.ffa_qk_norm_rope_axes(*{**AXES, **change}.values()) == code
    if not set(change) & {"qo", "ko"}:
        assert lib.ffa_qk_norm_rope_axes_bwd(*{**AXES_BWD, **change}.values()) == code


def test_norm_rope_axes_is_taken(lib):  # noqa: F811
    good = (OK, INVALID, UNSUPPORTED, OVERFLOW)
    bare = dict(qw=None, kw=None)
    for change in (dict(), bare, dict(n=4), dict(n=1, pairs=None), dict(n=1, pairs=None, **bare)):
        assert lib.ffa_qk_norm_rope_axes(*{**AXES, **change}.values()) not in good
        assert lib.ffa_qk_norm_rope_axes_bwd(*{**AXES_BWD, **change}.values()) not in good
    none = dict(q=None, k=None, dqw=None, dkw=None, ws=None, ws_bytes=0)
    assert lib.ffa_qk_norm_rope_axes_bwd(*{**AXES_BWD, **bare, **none}.values()) not in good
    assert lib.ffa_qk_norm_rope_axes_bwd(*{**AXES_BWD, **none}.values()) == INVALID
    # positions of all three axes are what outputs must not overlap
    assert lib.ffa_qk_norm_rope_axes(*{**AXES, "pos": at(6) - 32}.values()) == INVALID
    assert lib.ffa_qk_norm_rope_axes(*{**AXES, "pos": at(6) - 48}.values()) not in good


APPEND = dict(q=at(0), qs=512, k=at(1), ks=256, v=at(2), vs=256, tokens=4, hq=4, qw=at(3), kw=at(4), eps=1e-6, table=at(5), max_pos=16, rot=128,
              inter=0, pos=at(6), n=1, pairs=None, slots=at(7), cache=None, qo=at(8), stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID), (dict(hq=0), INVALID), (dict(rot=8), UNSUPPORTED), (dict(max_pos=0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(pos=None), INVALID),
    (dict(slots=None), INVALID), (dict(qo=None), INVALID), (dict(slots=at(7) + 4), INVALID), (dict(v=at(2) + 8), INVALID), (dict(vs=248), INVALID),
    (dict(vs=260), INVALID), (dict(qs=504), INVALID), (dict(n=0), INVALID), (dict(n=2), INVALID), (dict(n=5, pairs=ctypes.cast(PAIRS, ctypes.c_void_p)), UNSUPPORTED),
    (dict(qw=None), INVALID), (dict(qo=at(0)), INVALID), (dict(qo=at(2) + 64), INVALID), (dict(qo=at(20)), INVALID), (dict(v=at(21)), INVALID),
    (dict(slots=at(23)), INVALID), (dict(pos=at(24)), INVALID), (dict(qo=at(25)), INVALID), (dict(tokens=0, q=None, k=None, v=None, slots=None, qo=None, pos=None), OK),
    (dict(tokens=1 << 37), OVERFLOW)])
def test_append_refusals(lib, change, code):  # noqa: F811
    assert lib.ffa_kv_cache_append(*{**APPEND, "cache": ctypes.byref(cache4()), **change}.values()) == code


def test_append_is_taken_over_every_cache(lib):  # noqa: F811
    good = (OK, INVALID, UNSUPPORTED, OVERFLOW)
    for c in (cache(), cache4(), cache(dtype=0, k_exp=None, v_exp=None)):
        for change in (dict(), dict(qw=None, kw=None), dict(n=3, pairs=ctypes.cast(PAIRS, ctypes.c_void_p)), dict(inter=1)):
            assert lib.ffa_kv_cache_append(*{**APPEND, "cache": ctypes.byref(c), **change}.values()) not in good
    for c in (cache(dtype=2), cache(page_size=48)):
        assert lib.ffa_kv_cache_append(*{**APPEND, "cache": ctypes.byref(c)}.values()) == UNSUPPORTED
    assert lib.ffa_kv_cache_append(*{**APPEND, "cache": None}.values()) == INVALID


def test_binding_refuses_tensors_that_are_not_on_the_gpu(lib):  # noqa: F811
    import torch
    import flexible_mask_flashattention_gb300 as ffa
    x, w, t = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(4, 64)
    pos, c = torch.zeros(2, dtype=torch.int32), torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ffa.FFAError):
        ffa.kv_cache_append(x, x, x, w, w, t, pos, c, c, pos.long())


def test_axes_of_the_pairs_as_bytes():
    import torch
    from flexible_mask_flashattention_gb300 import FFAError, _lib
    want = bytes([0, 1, 2, 3])
    for axes in (want, [0, 1, 2, 3], (0, 1, 2, 3), range(4), np.arange(4), np.arange(4, dtype=np.uint8), torch.arange(4), bytearray(want)):
        assert _lib._pair_axes(axes) == want
    for bad in (4, np.int64(4), None, [0.5], [-1], [256], "01", [None], np.array([0.0, 1.0])):
        with pytest.raises(FFAError):
            _lib._pair_axes(bad)
