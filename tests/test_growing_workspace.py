"""How the 8-bit calls' own workspaces grow and let go (CPU: buffers of host
memory, the device's synchronisation and capture state stood in for)."""
import gc
import weakref

import pytest
import torch

import paged_kv_cache_139_gb300 as pkv


class World:
    def __init__(self, monkeypatch):
        self.capturing, self.synced, self.refs, self.most, self.room = False, 0, [], 0, 1 << 62
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: setattr(self, "synced", self.synced + 1))
        self.ws = pkv.GrowingWorkspace(self.make)

    def make(self, n):
        if self.held() + n > self.room:
            raise torch.OutOfMemoryError("no room")
        buf = torch.empty(n, dtype=torch.uint8)
        self.refs.append(weakref.ref(buf))
        self.most = max(self.most, self.held())
        return buf

    def held(self):
        gc.collect()
        return sum(r().numel() for r in self.refs if r() is not None)


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def test_a_prompt_in_chunks_holds_one_workspace(world):
    for n in range(8000, 512001, 8000):
        assert world.ws.get(n).numel() >= n
    assert world.held() <= 512000 * 3 // 2 and world.most <= 512000 * 3 // 2
    made = len(world.refs)
    assert made <= 12 and world.synced == made - 1                # 1.5 ** 11 > 64
    world.ws.get(100)
    assert len(world.refs) == made


def test_a_single_call_takes_what_it_needs(world):
    assert world.ws.get(1000).numel() == 1000 and world.synced == 0


def test_a_step_that_uses_the_old_one_keeps_it(world):
    old = world.ws.get(1000)
    new = world.ws.get(2000)
    assert old.numel() == 1000 and new.numel() == 2000 and old is not new


def test_a_captured_workspace_stays(world):
    world.ws.get(1000)
    world.capturing = True
    first = weakref.ref(world.ws.get(900))
    world.capturing = False
    for n in (2000, 4000, 9000):
        world.ws.get(n)
    gc.collect()
    assert first() is not None and sum(r() is not None for r in world.refs) == 2


def test_it_does_not_grow_during_a_capture(world):
    world.ws.get(1000)
    world.capturing = True
    with pytest.raises(RuntimeError, match="capture"):
        world.ws.get(1001)
    assert world.ws.get(1000).numel() == 1000
    world.capturing = False
    assert world.ws.get(1001).numel() == 1500


def test_short_of_memory_it_grows_by_what_is_needed(world):
    world.ws.get(1000)
    world.room = 1200
    assert world.ws.get(1100).numel() == 1100
    with pytest.raises(torch.OutOfMemoryError):
        world.ws.get(1201)
    world.room = 5000
    assert world.ws.get(3000).numel() == 3000


def test_another_streams_capture_counts(world, monkeypatch):
    import contextlib

    @contextlib.contextmanager
    def on(stream):
        was, world.capturing = world.capturing, stream == "captured"
        yield
        world.capturing = was

    monkeypatch.setattr(torch.cuda, "stream", on)
    world.ws.get(1000, stream="plain")
    with pytest.raises(RuntimeError):
        world.ws.get(2000, stream="captured")
    kept = weakref.ref(world.ws.get(1000, stream="captured"))
    world.ws.get(2000)
    gc.collect()
    assert kept() is not None


F8 = torch.float8_e4m3fn


def _cache(dtype=F8, device="cpu", **kw):
    from paged_kv_cache_139_gb300.engine import PagedKVCache
    return PagedKVCache(4, 2, 64, 16, dtype, device, 4, **kw)


def test_the_caches_of_a_models_layers_share_a_workspace(world):
    first = _cache()
    first._ws8 = world.ws
    layers = [first] + [_cache(workspace_of=first) for _ in range(3)]
    for n in (1000, 5000):
        bufs = [layer._workspace(n) for layer in layers]
        assert all(b is bufs[0] for b in bufs)
        del bufs
    assert world.held() == 5000
    assert _cache()._ws8 is not first._ws8


def test_what_cannot_share_a_workspace_is_refused():
    with pytest.raises(ValueError):
        _cache(workspace_of=_cache(torch.float16))
    with pytest.raises(ValueError):
        _cache(torch.float16, workspace_of=_cache())
    with pytest.raises(ValueError):
        _cache(torch.float16, workspace_of=_cache(torch.float16))
    with pytest.raises(ValueError):
        _cache(device="meta", workspace_of=_cache())


class Library:
    """pkv_check fails once with these flags; preparations are written down."""

    def __init__(self, flags):
        self.flags, self.prepared = flags, []

    def pkv_check(self, stream):
        return 5 if self.flags == 8 else 3

    def pkv_last_error_string(self):
        return b"device error flags 0x%x; first: something (value 1)" % self.flags

    def _init(self, ptr, nbytes, stream):
        self.prepared.append((ptr, nbytes))
        return 0

    paged_attention_workspace_init = paged_attention_fp8_workspace_init = _init


@pytest.mark.parametrize("flags,again", [(8, True), (8 | 2, True), (2, False), (128, False)])
def test_after_a_timeout_all_workspaces_are_prepared_again(monkeypatch, flags, again):
    import types
    stream = types.SimpleNamespace(cuda_stream=0, synchronize=lambda: None)
    synced = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)         # where the CPU's tensors say that they are
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: synced.append(len(lib.prepared)))
    monkeypatch.setattr(pkv, "_raw_stream", lambda s, index: 0)
    monkeypatch.setattr(pkv, "_workspaces", [])
    lib = Library(flags)
    monkeypatch.setattr(pkv, "load", lambda: lib)
    kept = [pkv.make_workspace("cpu", 1000), pkv.make_fp8_workspace("cpu", 2000)]
    pkv.make_fp8_workspace("cpu", 3000)                                   # gone
    lib.prepared.clear()
    gc.collect()
    with pytest.raises(pkv.PkvError):
        pkv.check()
    assert lib.prepared == ([(w.data_ptr(), w.numel()) for w in kept] if again else [])
    assert synced == ([0, 2] if again else [])
