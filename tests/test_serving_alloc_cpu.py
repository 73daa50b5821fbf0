"""The serving calls' way to new tensors: torch's quick allocation call is taken only where it gives what torch.empty_strided does."""
import pytest


def quick(change=None):
    import torch

    def make(size, strides, dtype):
        if change == "raises":
            raise TypeError("takes 4 positional arguments")
        if change == "no tensor":
            return 7
        t = torch.empty_strided(size, strides, dtype=torch.uint8 if change == "dtype" else dtype)
        return t.t() if change == "strides" else t[:1] if change == "size" else t

    return make


@pytest.mark.parametrize("change", ["raises", "no tensor", "dtype", "strides", "size"])
def test_an_allocation_call_that_does_something_else_is_not_taken(change):
    from flexible_mask_flashattention_gb300 import _lib
    assert _lib._gives_tensors(quick(), "cpu")
    assert not _lib._gives_tensors(quick(change), "cpu")
    assert not _lib._gives_tensors(None, "cpu")
    assert not _lib._gives_tensors(quick(), "cuda")


def test_start_finds_a_way_without_torchs_private_calls(monkeypatch):
    import torch
    from flexible_mask_flashattention_gb300 import _lib
    monkeypatch.delattr(torch._C._dynamo.guards, "_empty_strided_cuda", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    for name in ("torch", "_new", "_raw_stream"):
        monkeypatch.setattr(_lib, name, None)
    _lib._start()
    assert _lib._new is _lib._new_plain
    seen = []
    monkeypatch.setattr(torch, "empty_strided", lambda size, strides, dtype, device: seen.append((size, strides, dtype, device)))
    _lib._new((2, 3), (3, 1), torch.float32)
    assert seen == [((2, 3), (3, 1), torch.float32, "cuda")]

    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    assert _lib._raw_stream(0) == 77
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert _lib._gives_streams(lambda device: 77) and not _lib._gives_streams(lambda device: 78) and not _lib._gives_streams(None)


def test_deterministic_mode_allocates_with_torchs_own_call(monkeypatch):
    import torch
    from flexible_mask_flashattention_gb300 import _lib
    if _lib._new is None:
        _lib._start()
    monkeypatch.setattr(_lib, "_new", lambda *a: "quick")
    monkeypatch.setattr(_lib, "_new_plain", lambda *a: "plain")
    assert _lib._empty(None, (2, 3, 4), torch.float32) == "quick"
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        assert _lib._empty(None, (2, 3, 4), torch.float32) == "plain"
    finally:
        torch.use_deterministic_algorithms(was)


def test_interleaved_may_be_any_truth_value(monkeypatch):
    import ctypes
    import numpy as np
    import torch
    from flexible_mask_flashattention_gb300 import _lib
    got = []

    class Library:
        def ffa_qk_norm_rope(self, *args):
            got.append(ctypes.c_int32(args[14]).value)
            return 0

        def ffa_qk_norm_rope_bwd(self, *args):
            got.append(ctypes.c_int32(args[14]).value)
            return 0

        def ffa_qk_norm_rope_bwd_workspace_size(self, d):
            return 16

    monkeypatch.setattr(_lib, "torch", torch)
    monkeypatch.setattr(_lib, "load_library", Library)
    monkeypatch.setattr(_lib, "_device", lambda t, name: -1)
    monkeypatch.setattr(_lib, "_on", lambda *a: (0, None))
    monkeypatch.setattr(_lib, "_empty", lambda context, size, dtype: torch.empty(size, dtype=dtype))
    x, w, t, pos = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(4, 64), torch.zeros(2, dtype=torch.int32)
    for value in (True, np.bool_(True), torch.tensor(True), 2):
        _lib.qk_norm_rope(x, x, w, w, t, pos, interleaved=value)
        _lib.qk_norm_rope_bwd(x, x, w, w, t, pos, x, x, interleaved=value)
    assert got == [1] * 8
