"""Whose device the scratch of decode over shared prefixes is sized for (no GPU:
devices and the library are stood in for)."""
import contextlib
import types

import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from paged_kv_cache_139_gb300 import engine

SIZES = (4, 1, 8, 8, 64, 300, 260, 4, 40)


@pytest.fixture
def devices(monkeypatch):
    """Two devices whose plans need 1000 and 2000 bytes; state.now is the current one."""
    state = types.SimpleNamespace(now=0, asked=[])

    @contextlib.contextmanager
    def device(index):
        was, state.now = state.now, index
        yield
        state.now = was

    def size(*sizes):
        state.asked.append((state.now, sizes))
        return 1000 * (state.now + 1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.now)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "device", device)
    lib = types.SimpleNamespace(paged_attention_decode_shared_workspace_size=size, paged_attention_decode_shared=lambda *a: 0)
    monkeypatch.setattr(pkv, "load", lambda: lib)
    yield state
    if hasattr(pkv, "_shared_size_on"):
        pkv._shared_size_on.cache_clear()


def test_the_current_devices_size(devices):
    size = pkv.paged_attention_decode_shared_workspace_size
    assert size(*SIZES) == 1000
    devices.now = 1
    assert size(*SIZES) == 2000
    devices.now = 0
    assert size(*SIZES) == 1000 and devices.asked == [(0, SIZES), (1, SIZES)]


def test_a_named_devices_size_on_another_one(devices):
    assert pkv.paged_attention_decode_shared_workspace_size(*SIZES, 1) == 2000 and devices.now == 0


def test_the_bindings_scratch_is_sized_on_the_tensors_device(devices, monkeypatch):
    """The tensors lie on device 1, device 0 is current."""
    need = []
    monkeypatch.setattr(pkv, "_check16", lambda *a: (1, (0,) * 6, 2, (8, 2, 16, 64)))
    monkeypatch.setattr(pkv, "_at", lambda t, *a: 0)
    monkeypatch.setattr(pkv, "_call", lambda fn, what, index, *args: fn(*args))
    monkeypatch.setattr(pkv, "_raw_stream", lambda s, index: 0)
    monkeypatch.setattr(pkv, "_scratch", lambda index, n, stream: need.append((index, n)) or torch.zeros(1, dtype=torch.uint8))
    q, i32 = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    pkv.paged_attention_decode_shared(q, q, q, q, q, i32, torch.zeros(2, dtype=torch.int32), i32)
    assert need == [(1, 2000)]


def test_a_prepared_steps_scratch_is_sized_on_the_caches_device(devices, monkeypatch):
    groups = engine.DeviceGroups(torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 260, 4, 40)
    eng = types.SimpleNamespace(num_kv_heads=8, device="cpu", key_cache=types.SimpleNamespace(get_device=lambda: 1))
    assert engine._scratch_shared(eng, groups, 4, 8, 64, 300, None).numel() == 2000
