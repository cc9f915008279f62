"""The binding's host side, without a GPU."""
from __future__ import annotations

import threading

import pytest

torch = pytest.importorskip("torch")

from mixed_precision_dense_02_gb300 import binding


def test_tensor_types_are_complete_for_every_thread(monkeypatch):
    """A thread that asks for the types while another one is putting them
    together gets all of them."""
    seen = []

    class Slow:
        """torch, where looking up an 8-bit type lets another thread run."""

        def __getattr__(self, name):
            if name == "float8_e4m3fn" and threading.current_thread() is threading.main_thread():
                t = threading.Thread(target=lambda: seen.append(set(binding._kinds())))
                t.start()
                t.join()
            return getattr(torch, name)

    monkeypatch.setattr(binding, "_KIND", {})
    monkeypatch.setattr(binding, "_torch", Slow)
    every = {"wide", "half", "f8", "scale", "offset", "fmt"}
    assert set(binding._kinds()) == every
    assert seen and all(s == every for s in seen)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device; tensors of another one are
    refused on every call, a plan kept from an earlier call or not."""
    class Fake:
        class _C:
            _cuda_getDevice = staticmethod(lambda: 1)
            _cuda_getCurrentRawStream = staticmethod(lambda index: 7)

    monkeypatch.setattr(binding, "_torch", lambda: Fake)
    assert binding._raw_stream(1) == 7
    with pytest.raises(ValueError, match="cuda:0"):
        binding._raw_stream(0)


def test_abort_selftest_arguments():
    from mixed_precision_dense_02_gb300 import build
    build.build()
    p, ok, invalid, misaligned, nodev = 1 << 20, 0, 1, 3, 6
    f = binding.mma_selftest_f8_abort
    assert f(-1, 10 ** 7, p, p, p, None, None) == f(6, 10 ** 7, p, p, p, p, None) == invalid
    assert f(0, 10, p, p, p, None, None) == f(1, 10 ** 11, p, p, p, None, None) == invalid
    assert f(0, 10 ** 7, None, p, p, None, None) == f(2, 10 ** 7, p, p, p, None, None) == invalid
    assert f(0, 10 ** 7, p, p + 8, p, None, None) == misaligned
    if not torch.cuda.is_available():  # (these addresses are fake)
        assert f(0, 10 ** 7, p, p, p, None, None) == f(2, 10 ** 7, p, p, p, p, None) == nodev
        assert f(3, 10 ** 7, p, p, p, None, None) == f(5, 10 ** 7, p, p, p, None, None) == nodev
