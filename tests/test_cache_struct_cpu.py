"""A cache description without the fields of the 4-bit type, as a program has that was compiled before they were there: the calls read none of what
lies behind it.  The description ends where a mapped page ends, the next page cannot be read, so that a call that does ends its process."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import ctypes, mmap, sys
import flexible_mask_flashattention_gb300 as ffa
from flexible_mask_flashattention_gb300._lib import KVCacheC
lib = ffa.load_library()
libc = ctypes.CDLL(None, use_errno=True)
libc.mmap.restype = ctypes.c_void_p
libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long]
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
page = mmap.PAGESIZE
base = libc.mmap(None, 2 * page, mmap.PROT_READ | mmap.PROT_WRITE, mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS, -1, 0)
assert base not in (None, ctypes.c_void_p(-1).value) and libc.mprotect(base + page, page, 0) == 0
at = lambda i: (1 << 32) + (i << 24)   # never read: no GPU can be seen
dtype, size, what = int(sys.argv[1]), KVCacheC.k_scale.offset, sys.argv[2]
exps = (at(22), at(23)) if dtype else (None, None)
c = KVCacheC(at(20), at(21), *exps, 10, 64, 2, 128, dtype, None, None)
where = base + page - size
ctypes.memmove(where, ctypes.byref(c), size)
calls = dict(
    write=lambda: lib.ffa_kv_cache_write(at(0), 256, at(1), 512, 3, at(2), where, None),
    read=lambda: lib.ffa_kv_cache_read(where, at(0), 4, 4, 2, at(1), 7, at(2), at(3), None),
    decode=lambda: lib.ffa_fwd_decode(at(0), 512, where, at(1), 4, 4, 2, 4, at(2), None, 0.1, None, at(3), at(4), at(5), 1 << 30, None),
    window=lambda: lib.ffa_fwd_decode_window(at(0), 512, where, at(1), 4, 4, 2, 4, at(2), None, at(9), 0.1, None, at(3), at(4), at(5), 1 << 30, None),
    append=lambda: lib.ffa_kv_cache_append(at(0), 512, at(1), 256, at(2), 256, 4, 4, at(3), at(4), 1e-6, at(5), 16, 128, 0, at(6), 1, None, at(7),
                                           where, at(8), None))
print("status", calls[what]())
"""


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("what", ["write", "read", "decode", "window", "append"])
def test_nothing_behind_the_older_description_is_read(what, dtype):
    from flexible_mask_flashattention_gb300 import build
    build.build()
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": "", "PYTHONPATH": ROOT}
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(dtype), what], env=env, capture_output=True, text=True, timeout=120, cwd=ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.split() == ["status", "6"]   # past every check, as far as CUDA
