"""A 4-bit cache is used on the device it lives on: with another current device
the binding refuses the call instead of handing the kernel an address that
the device does not have (CPU only: stand-ins for tensors of two devices, and
a library that records what reaches it)."""

import pytest
import torch

from lossless_draft_verify_vc_b200 import vc


class Fake:
    def __init__(self, dev, dtype, *shape):
        self.dev, self.dtype, self.shape = dev, dtype, shape

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 0x10000


class Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def two(monkeypatch):
    """Current device 0, then whatever the test sets."""
    now, L = [0], Lib()
    monkeypatch.setattr(vc, "_device", lambda: now[0])
    monkeypatch.setattr(vc, "_raw_stream", lambda d: 0)
    monkeypatch.setattr(vc, "lib", lambda: L)
    return now, L


def calls(fc, dev):
    sh = vc.shape(1, 4, 2, 64)
    x = Fake(dev, torch.bfloat16, 1, 2, 3, 64)
    ws = Fake(dev, torch.uint8, 1 << 20)
    q, out = Fake(dev, torch.bfloat16, 1, 4, 64), Fake(dev, torch.float32, 1, 4, 64)
    return [lambda: vc.vc_fp4_cache_write(sh, fc, x, x, 3, ws), lambda: vc.vc_fp4_cache_read(sh, fc, 3, x, x, ws),
            lambda: vc.vc_draft_attn_fp4(sh, fc, q, out, ws)]


def test_a_cache_of_another_device_is_refused(two):
    now, L = two
    fc = vc.fp4_cache(Fake(0, torch.uint8, 1, 2, 4, 18 * 64))
    now[0] = 1
    for call in calls(fc, 1):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not L.calls


def test_tensors_of_another_device_are_refused(two):
    now, L = two
    fc = vc.fp4_cache(Fake(0, torch.uint8, 1, 2, 4, 18 * 64))
    for call in calls(fc, 1):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    assert not L.calls


def test_its_own_device_passes(two):
    now, L = two
    now[0] = 1
    fc = vc.fp4_cache(Fake(1, torch.uint8, 1, 2, 4, 18 * 64))
    for call in calls(fc, 1):
        call()
    assert L.calls == ["vc_fp4_cache_write", "vc_fp4_cache_read", "vc_draft_attn_fp4"]


def test_a_descriptor_of_raw_pointers_passes(two):
    now, L = two
    now[0] = 1
    for call in calls(vc.vc_fp4_cache(0x10000, 64, 64, 0, 0, 0), 1):
        call()
    assert len(L.calls) == 3
