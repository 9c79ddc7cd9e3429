"""On which stream the bindings take the memory that they give to a call (CPU:
streams, allocations and the library are stood in for)."""
import contextlib
import gc
import types
import weakref

import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from paged_kv_cache_139_gb300 import engine

STREAM = types.SimpleNamespace(cuda_stream=77, synchronize=lambda: None)


class Library:
    """Every call succeeds and is written down."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    """Tensors on the CPU pass for CUDA ones; made: (size, current stream) of every uninitialised tensor."""
    stack, made, recorded = [None], [], []

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream)
        yield
        stack.pop()

    def watched(make):
        def empty(*args, **kw):
            kw.pop("device", None)
            t = make(*args, **kw)
            made.append((tuple(t.shape), stack[-1]))
            return t
        return empty

    lib = Library()
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch, "empty", watched(torch.empty))
    monkeypatch.setattr(torch, "empty_like", watched(torch.empty_like))
    monkeypatch.setattr(pkv, "load", lambda: lib)
    monkeypatch.setattr(engine, "load", lambda: lib)
    monkeypatch.setattr(pkv, "_cuda_index", lambda t, name: t.get_device())
    monkeypatch.setattr(pkv, "_call", lambda fn, what, index, *args: fn(*args))
    return types.SimpleNamespace(made=made, lib=lib, recorded=recorded)


def _tokens():
    z = lambda *shape: torch.zeros(*shape, dtype=torch.float16)  # noqa: E731
    return z(3, 4, 64), z(3, 2, 64), z(3, 2, 64)


@pytest.mark.parametrize("stream", [None, STREAM])
@pytest.mark.parametrize("fp8", [False, True])
def test_rotated_queries_are_made_on_the_calls_stream(world, monkeypatch, stream, fp8):
    monkeypatch.setattr(pkv, "_raw_stream", lambda s, index: 0 if s is None else s.cuda_stream)
    q, k, v = _tokens()
    cs, pos, slots = torch.zeros(10, 32, 2), torch.zeros(3, dtype=torch.int32), torch.arange(3)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn if fp8 else torch.float16)
    if fp8:
        out = pkv.kv_rotary_and_cache_fp8(q, k, v, cs, pos, kc, kc.clone(), torch.zeros(4, 2, 2), slots, stream=stream)
    else:
        out = pkv.kv_rotary_and_cache(q, k, v, cs, pos, kc, kc.clone(), slots, stream=stream)
    assert out.shape == q.shape and world.made == [((3, 4, 64), stream)]
    assert world.lib.calls[0][1][-1] == (77 if stream else 0)


@pytest.mark.parametrize("stream", [None, STREAM])
def test_tables_and_workspaces_are_made_on_the_calls_stream(world, monkeypatch, stream):
    monkeypatch.setattr(pkv, "_raw_stream", lambda s, index: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0, synchronize=lambda: None))
    pkv.rotary_table(10, 64, device="cpu", stream=stream)
    pkv.make_workspace("cpu", 1000, stream=stream)
    pkv.make_fp8_workspace("cpu", 2000, stream=stream)
    assert world.made == [((10, 32, 2), stream), ((1000,), stream), ((2000,), stream)]


def _engine(monkeypatch, fp8, rotary):
    monkeypatch.setattr(engine, "_check_step", lambda *a, **k: 0)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    monkeypatch.setattr(engine.PagedKVCache, "_workspace", lambda self, need: ws)
    monkeypatch.setattr(engine.PagedKVCache, "workspace", lambda self, *a: ws)
    monkeypatch.setattr(engine.PagedKVCache, "prefill_workspace", lambda self: ws)
    monkeypatch.setattr(engine, "BlockAllocator", lambda *a: None)
    monkeypatch.setattr(engine, "paged_attention_prefill_fp8_workspace_size", lambda *a: 0)
    cs = engine.RotaryPositions(torch.zeros(10, 32, 2)) if rotary else None
    eng = engine.PagedKVCache(4, 2, 64, 16, torch.float8_e4m3fn if fp8 else torch.float16, "cpu", 4, rotary=cs)
    return eng, ws


def _step(kind):
    e = torch.zeros(0, 2, dtype=torch.int32)
    common = dict(slots=torch.arange(3), pairs=e, tables=torch.zeros(3, 4, dtype=torch.int32),
                  context_lens=torch.ones(3, dtype=torch.int32), positions=torch.zeros(3, dtype=torch.int32), max_context_len=1)
    if kind == "prefill":
        return engine.DevicePrefill(query_start=torch.arange(4, dtype=torch.int32), max_query_len=1, **common)
    return engine.DeviceStep(**common)


def _prepare(eng, kind, stream=STREAM):
    q, k, v = _tokens()
    out = torch.zeros_like(q)
    prepare = eng.prepare_prefill if kind == "prefill" else eng.prepare
    return prepare(q, k, v, _step(kind), out, stream=stream)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_prepared_step_takes_its_queries_scratch_on_its_stream(world, monkeypatch, kind, fp8):
    eng, ws = _engine(monkeypatch, fp8, rotary=True)
    world.made.clear()
    step = _prepare(eng, kind)
    assert world.made == [((3, 4, 64), STREAM)] and (ws.data_ptr(), STREAM) in world.recorded
    assert dict(world.lib.calls) == {}
    step()
    assert len(world.lib.calls) == 2


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("fp8,rotary", [(False, False), (False, True), (True, False), (True, True)])
def test_a_prepared_step_keeps_what_it_reads(world, monkeypatch, kind, fp8, rotary):
    """The pools, the scales and the table that its calls address, whatever the cache holds by then."""
    eng, _ = _engine(monkeypatch, fp8, rotary)
    step = _prepare(eng, kind)
    tensors = [t for t in (eng.key_cache, eng.value_cache, eng.scales, eng.rotary and eng.rotary.cos_sin) if t is not None]
    assert all((t.data_ptr(), STREAM) in world.recorded for t in tensors)
    held = [weakref.ref(t) for t in tensors]
    del tensors
    if rotary:
        eng.rotary = engine.RotaryPositions(torch.zeros(20, 32, 2))
    eng.key_cache = eng.value_cache = eng.scales = None
    del eng
    gc.collect()
    assert len(held) == 2 + fp8 + rotary and all(r() is not None for r in held)
    del step
    gc.collect()
    assert all(r() is None for r in held)


@pytest.mark.parametrize("fp8,rotary", [(False, True), (True, False), (True, True)])
def test_the_fused_write_serves_plain_16_bit_caches_only(world, monkeypatch, fp8, rotary):
    eng, _ = _engine(monkeypatch, fp8, rotary)
    step = _prepare(eng, "decode")
    with pytest.raises(ValueError):
        step.write_attend()
    assert world.lib.calls == []
    step()
    assert [name for name, _ in world.lib.calls] == [
        "kv_rotary_and_cache" + ("_fp8" if fp8 else ""),
        "paged_attention_decode" + ("_fp8" if fp8 else "")]


def test_the_fused_write_takes_a_token_for_each_sequence(world, monkeypatch):
    """A plan without new tokens has no keys, values and slots for the fused call to read."""
    eng, _ = _engine(monkeypatch, False, False)
    step = _prepare(eng, "decode")
    step.write_attend()
    assert world.lib.calls[-1][0] == "paged_attention_decode_write"
    q, k, v = _tokens()
    none = _step("decode")
    none.slots = none.slots[:0]
    step = eng.prepare(q, k[:0], v[:0], none, torch.zeros_like(q), stream=STREAM)
    world.lib.calls.clear()
    with pytest.raises(ValueError):
        step.write_attend()
    step()
    assert [name for name, _ in world.lib.calls] == ["paged_attention_decode"]


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("wrong", [lambda x: x.long(), lambda x: x[:2], lambda x: None, lambda x: x.repeat_interleave(2)[::2]])
def test_prepared_steps_refuse_positions_that_are_not_32_bit_ones(monkeypatch, kind, wrong):
    """The eager calls refuse them; a prepared step hands on addresses and would read other numbers."""
    check = engine._check_step
    eng, _ = _engine(monkeypatch, False, True)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    q, k, v = _tokens()
    step = _step(kind)
    assert check(eng, q, k, v, step, torch.zeros_like(q)) == 0
    step.positions = wrong(step.positions)
    with pytest.raises(AssertionError):
        check(eng, q, k, v, step, torch.zeros_like(q))


@pytest.mark.parametrize("table", [torch.zeros(10, 32, 2).double(), torch.zeros(10, 64), torch.zeros(10, 32, 4)[..., :2],
                                   torch.zeros(10, 32, 2, device="meta")])
def test_prepared_steps_refuse_tables_of_another_kind(monkeypatch, table):
    check = engine._check_step
    eng, _ = _engine(monkeypatch, False, True)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    eng.rotary = engine.RotaryPositions(table)
    q, k, v = _tokens()
    with pytest.raises(AssertionError):
        check(eng, q, k, v, _step("decode"), torch.zeros_like(q))


def test_caches_refuse_scales_and_pools_of_another_kind():
    f8 = torch.float8_e4m3fn
    pool = torch.zeros(4, 3, 16, 64).to(f8)
    make = lambda **kw: engine.PagedKVCache(4, 3, 64, 16, f8, "cpu", 4, **kw)  # noqa: E731
    make(key_cache=pool, value_cache=pool.clone(), scales=torch.zeros(4, 4, 2))
    for bad in (torch.zeros(4, 3, 2), torch.zeros(3, 4, 2), torch.zeros(4, 4, 2).double(), torch.zeros(4, 2, 4).transpose(1, 2)):
        with pytest.raises(AssertionError):
            make(scales=bad)
    with pytest.raises(AssertionError):
        make(key_cache=torch.zeros(4, 3, 16, 64, dtype=torch.float16))
    with pytest.raises(AssertionError):
        make(value_cache=torch.zeros(4, 3, 64, 16).to(f8).transpose(2, 3))


def test_swaps_keep_their_pairs_until_their_copies_are_done(monkeypatch):
    """Several swaps may be issued before the first one's copies have read their pairs."""
    import numpy as np
    events = []

    class Event:
        def __init__(self):
            self.done, self.stream = False, None
            events.append(self)

        def record(self, stream):
            self.stream = stream

        def query(self):
            return self.done

    alive, copied = [], []
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: alive.append(weakref.ref(c := t.clone())) or c)
    monkeypatch.setattr(engine, "swap_blocks", lambda dst, src, pairs, stream: copied.append(pairs.data_ptr()))
    eng = engine.PagedKVCache(4, 2, 64, 16, torch.float8_e4m3fn, "cpu", 4)
    move = lambda *a: ([0], np.zeros((2, 2), np.int32))  # noqa: E731
    eng.alloc = types.SimpleNamespace(move_group=move)
    host = types.SimpleNamespace(key_cache=None, value_cache=None, scales=torch.zeros(1), alloc=eng.alloc)
    held = lambda: gc.collect() and None or [r() is not None for r in alive]  # noqa: E731
    eng.swap_out([0], host)
    eng.swap_in([0], host, stream=STREAM)
    eng.swap_out([0], host)
    assert held() == [True] * 3 and [e.stream for e in events] == ["current", STREAM, "current"] and len(copied) == 9
    events[0].done = events[1].done = True
    eng.swap_in([0], host)
    assert held() == [False, False, True, True]


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_a_prepared_step_marks_what_it_holds_on_the_current_stream(world, monkeypatch, kind):
    """Without a stream of its own; the pools and the workspace may come from another."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: STREAM)
    eng, ws = _engine(monkeypatch, True, True)
    _prepare(eng, kind, stream=None)()
    held = {t.data_ptr() for t in (ws, eng.key_cache, eng.value_cache, eng.scales, eng.rotary.cos_sin)}
    assert {p for p, s in world.recorded if s is STREAM} == held
    assert all(args[-1].value == 77 for _, args in world.lib.calls)
