"""Windowed and shared-prefix attention on the host: refusals through the C ABI
and the bindings, workspace sizes, the groups of a step, what the engine calls
(no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from paged_kv_cache_139_gb300 import engine
from paged_kv_cache_139_gb300._lib import load
from test_streams_host import STREAM, _tokens, world  # noqa: F401  (fixture)

P = 1 << 20                     # an aligned address that is never read: every call here is refused or has nothing to do


def call(name, base, over):
    args = {**base, **over}
    return getattr(load(), name)(*args.values())


def message():
    return load().pkv_last_error_string().decode()


WINDOW = dict(out=P, q=P, kc=P, vc=P, bt=P, cl=P, S=2, mb=4, mcl=0, B=16, NB=8, H=4, Hkv=2, d=128, scale=0.1, window=8, sinks=2,
              dt=0, st=None)
PROMPT = dict(out=P, q=P, kc=P, vc=P, bt=P, cl=P, qs=P, S=2, T=10, mql=0, mb=4, B=16, NB=8, H=4, Hkv=2, d=128, scale=0.1, window=8,
              sinks=2, ws=None, wsb=0, dt=0, st=None)
SHARED = dict(out=P, q=P, kc=P, vc=P, bt=P, cl=P, gs=P, pl=P, S=4, G=2, mgs=0, mpl=0, msl=0, mb=4, mcl=0, B=16, NB=8, H=4, Hkv=2,
              d=128, scale=0.1, ws=P, wsb=1 << 30, dt=0, st=None)
COMMON = [dict(d=96), dict(d=256), dict(d=0), dict(B=12), dict(B=2), dict(B=256), dict(B=0), dict(H=5), dict(H=0), dict(Hkv=0),
          dict(dt=2), dict(dt=-1), dict(S=-1), dict(S=65536), dict(mb=-1), dict(NB=-1), dict(out=None), dict(q=None), dict(kc=None),
          dict(vc=None), dict(bt=None), dict(cl=None), dict(out=24), dict(q=8), dict(kc=18), dict(vc=4),
          dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("over", COMMON + [dict(window=0), dict(window=-1), dict(sinks=-1), dict(mcl=65), dict(mcl=-1),
                                           dict(mb=(1 << 26) + 1), dict(H=65536, Hkv=1), dict(S=40000, H=32768, Hkv=1)])
def test_window_refusals(over):
    assert call("paged_attention_decode_window", WINDOW, over) == 1
    assert message().startswith("paged_attention_decode_window")


@pytest.mark.parametrize("over", COMMON + [dict(window=0), dict(sinks=-3), dict(T=-1), dict(mql=-1), dict(qs=None), dict(mb=0),
                                           dict(mb=1 << 28), dict(NB=0), dict(scale=0.0), dict(scale=-1.0), dict(ws=24, wsb=256),
                                           dict(ws=P, wsb=255)])
def test_prompt_refusals(over):
    assert call("paged_attention_prefill_window", PROMPT, over) == 1
    assert message().startswith("paged_attention_prefill_window")


@pytest.mark.parametrize("over", COMMON + [dict(G=0), dict(G=-1), dict(G=5), dict(mgs=-1), dict(mpl=-1), dict(msl=-1), dict(mpl=65),
                                           dict(gs=None), dict(pl=None), dict(ws=None), dict(ws=24), dict(wsb=100), dict(mcl=65),
                                           dict(scale=0.0), dict(scale=-0.5), dict(H=258, Hkv=2), dict(mb=(1 << 26) + 1)])
def test_shared_refusals(over):
    assert call("paged_attention_decode_shared", SHARED, over) == 1
    assert message().startswith("paged_attention_decode_shared")


def test_nothing_to_do():
    assert call("paged_attention_decode_window", WINDOW, dict(S=0)) == 0
    assert call("paged_attention_prefill_window", PROMPT, dict(S=0)) == 0
    assert call("paged_attention_prefill_window", PROMPT, dict(T=0)) == 0
    assert call("paged_attention_decode_shared", SHARED, dict(S=0, G=0)) == 0
    n = pkv.launch_count()
    assert n == pkv.launch_count()


def test_shared_workspace_sizes():
    size = pkv.paged_attention_decode_shared_workspace_size
    small = size(4, 1, 8, 8, 64, 300, 260, 4, 40)
    row = 4 * (64 + 2)                                   # a part of a row: its maximum, sum and values
    assert 4 * 8 * row <= small <= 3 * 4 * 8 * row + 1024        # one to three parts of each row
    # what a call with wider bounds needs is no less than with narrow ones of the same split
    assert size(4, 1, 8, 8, 64, 300) >= 4 * 8 * row
    big = size(128, 1, 32, 8, 128, 9216, 8192, 128, 1024)
    assert 128 * 32 * 4 * 130 * 2 <= big <= 128 * 32 * 4 * 130 * 80
    for bad in (dict(num_seqs=0), dict(num_groups=0), dict(num_heads=0), dict(num_kv_heads=0), dict(num_heads=5),
                dict(num_heads=258), dict(head_dim=0), dict(max_context_len=-1), dict(max_prefix_len=-1),
                dict(max_group_size=-1), dict(max_suffix_len=-1)):
        kw = {**dict(num_seqs=4, num_groups=1, num_heads=8, num_kv_heads=2, head_dim=64, max_context_len=300), **bad}
        assert size(**kw) == 0


def test_bindings_refuse_what_does_not_fit():
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)  # noqa: E731
    q, kc, bt, cl = z(3, 4, 64), z(8, 2, 16, 64), z(3, 2, dt=torch.int32), z(3, dt=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        pkv.paged_attention_decode_window(q, q, kc, kc, bt, cl, 4)
    with pytest.raises(TypeError, match="CUDA"):
        pkv.paged_attention_prefill_window(q, q, kc, kc, bt, cl, z(4, dt=torch.int32), 4)
    with pytest.raises(TypeError, match="CUDA"):
        pkv.paged_attention_decode_shared(q, q, kc, kc, bt, cl, z(2, dt=torch.int32), cl)


@pytest.fixture
def passes(world, monkeypatch):  # noqa: F811
    """CPU tensors pass for CUDA ones (device -1)."""
    monkeypatch.setattr(pkv, "_raw_stream", lambda s, index: 0 if s is None else s.cuda_stream)
    return world


def window_args(**over):
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)  # noqa: E731
    a = dict(out=z(3, 4, 64), query=z(3, 4, 64), key_cache=z(8, 2, 16, 64), value_cache=z(8, 2, 16, 64),
             block_tables=z(3, 2, dt=torch.int32), context_lens=z(3, dt=torch.int32))
    return {**a, **over}


@pytest.mark.parametrize("over,kind", [
    (dict(out=torch.zeros(3, 4, 32, dtype=torch.float16)), ValueError),
    (dict(out=torch.zeros(3, 4, 64)), TypeError),
    (dict(key_cache=torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)), TypeError),
    (dict(value_cache=torch.zeros(7, 2, 16, 64, dtype=torch.float16)), ValueError),
    (dict(key_cache=torch.zeros(8, 16, 2, 64, dtype=torch.float16).transpose(1, 2)), ValueError),
    (dict(query=torch.zeros(4, 3, 64, dtype=torch.float16).transpose(0, 1)), ValueError),
    (dict(block_tables=torch.zeros(3, 2, dtype=torch.int64)), TypeError),
    (dict(block_tables=torch.zeros(4, 2, dtype=torch.int32)), ValueError),
    (dict(block_tables=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(context_lens=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(context_lens=torch.zeros(6, dtype=torch.int32)[::2]), ValueError),
])
def test_bindings_check_shapes_types_and_strides(passes, monkeypatch, over, kind):
    def wrong(t, name, dtype=None, ndim=None):           # as _dev, for tensors of the CPU
        if not t.is_contiguous():
            raise ValueError(name)
        if dtype is not None and t.dtype != dtype:
            raise TypeError(name)
        return t.data_ptr()
    monkeypatch.setattr(pkv, "_dev", wrong)
    a = window_args(**over)
    with pytest.raises(kind):
        pkv.paged_attention_decode_window(**a, window=4)
    with pytest.raises(kind):
        pkv.paged_attention_prefill_window(**a, query_start=torch.zeros(4, dtype=torch.int32), window=4)
    with pytest.raises(kind):
        pkv.paged_attention_decode_shared(**a, group_start=torch.zeros(2, dtype=torch.int32),
                                          prefix_lens=torch.zeros(3, dtype=torch.int32), workspace=torch.zeros(1, dtype=torch.uint8))
    assert passes.lib.calls == []


def test_bindings_pass_their_arguments_on(passes):
    a = window_args()
    ptrs = tuple(a[k].data_ptr() for k in ("out", "query", "key_cache", "value_cache", "block_tables", "context_lens"))
    pkv.paged_attention_decode_window(**a, window=9, num_sinks=3, scale=0.5, max_context_len=30, stream=STREAM)
    qs = torch.zeros(4, dtype=torch.int32)
    pkv.paged_attention_prefill_window(**a, query_start=qs, window=9, num_sinks=3, scale=0.5, max_query_len=2)
    gs, pl, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(99, dtype=torch.uint8)
    pkv.paged_attention_decode_shared(**a, group_start=gs, prefix_lens=pl, scale=0.5, max_context_len=30, max_prefix_len=16,
                                      max_group_size=3, max_suffix_len=14, workspace=ws)
    assert passes.lib.calls == [
        ("paged_attention_decode_window", (*ptrs, 3, 2, 30, 16, 8, 4, 2, 64, 0.5, 9, 3, 0, 77)),
        ("paged_attention_prefill_window", (*ptrs, qs.data_ptr(), 3, 3, 2, 2, 16, 8, 4, 2, 64, 0.5, 9, 3, None, 0, 0, 0)),
        ("paged_attention_decode_shared", (*ptrs, gs.data_ptr(), pl.data_ptr(), 3, 1, 3, 16, 14, 2, 30, 16, 8, 4, 2, 64, 0.5,
                                           ws.data_ptr(), 99, 0, 0))]


def test_windows_beyond_32_bits_see_everything(passes):
    """ctypes would take the lower 32 bits."""
    a, qs = window_args(), torch.zeros(4, dtype=torch.int32)
    pkv.paged_attention_decode_window(**a, window=(1 << 32) + 5, num_sinks=(1 << 40) + 1)
    pkv.paged_attention_prefill_window(**a, query_start=qs, window=1 << 31, num_sinks=1 << 32)
    assert passes.lib.calls[0][1][15:17] == (2 ** 31 - 1,) * 2 and passes.lib.calls[1][1][17:19] == (2 ** 31 - 1,) * 2
    eng = engine.PagedKVCache(4, 2, 64, 16, torch.float16, "cpu", 4, window=1 << 40, sinks=1 << 33)
    assert (eng.window, eng.sinks) == (2 ** 31 - 1,) * 2
    passes.lib.calls.clear()
    for window, sinks in ((0, 0), (-(1 << 32) + 5, 0), (4, -1), (4, -(1 << 32) + 1)):
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_window(**a, window=window, num_sinks=sinks)
        with pytest.raises(ValueError):
            pkv.paged_attention_prefill_window(**a, query_start=qs, window=window, num_sinks=sinks)
    assert passes.lib.calls == []


# -- the groups of a step ------------------------------------------------------------------

def groups(rows, ctx, B=4):
    width = max(len(r) for r in rows)
    t = np.full((len(rows), width), -1, np.int32)
    for i, r in enumerate(rows):
        t[i, :len(r)] = r
    g = engine.SharedGroups.find(t, np.asarray(ctx, np.int32), B)
    return g.start.tolist(), g.prefix.tolist()


def test_groups_of_forks():
    assert groups([[1, 2, 3], [1, 2, 4], [1, 2, 5, 6]], [9, 10, 14]) == ([0, 3], [8, 8, 8])


def test_only_full_blocks_are_shared():
    assert groups([[1, 2], [1, 2]], [7, 7]) == ([0, 2], [4, 4])
    assert groups([[1, 2], [1, 2]], [8, 8]) == ([0, 2], [8, 8])
    assert groups([[1], [1]], [3, 4]) == ([0, 1, 2], [0, 0])


def test_strangers_and_single_sequences_share_nothing():
    assert groups([[1, 2], [3, 4], [5]], [8, 8, 4]) == ([0, 1, 2, 3], [0, 0, 0])
    assert groups([[1, 2]], [8]) == ([0, 1], [0])


def test_a_group_is_left_where_that_saves_more():
    """Two samples of a long prompt and another request that shares its first block only."""
    long = list(range(10, 20))
    assert groups([long + [1], long + [2], [10, 3]], [41, 41, 8]) == ([0, 2, 3], [40, 40, 0])
    # ... and where joining saves more: many sequences on one block
    assert groups([[1, 2, 9], [1, 2, 8], [1, 3], [1, 4], [1, 5]], [9, 9, 6, 6, 6])[0] == [0, 5]


def test_groups_of_nothing():
    g = engine.SharedGroups.find(np.zeros((0, 3), np.int32), np.zeros(0, np.int32), 4)
    assert g.start.tolist() == [0] and g.prefix.size == 0


def test_random_groups_are_what_they_say():
    rng = np.random.default_rng(0)
    for _ in range(200):
        n, w = int(rng.integers(1, 9)), int(rng.integers(1, 6))
        t = np.minimum(rng.integers(0, 3, (n, w)), rng.integers(0, 3)).astype(np.int32)
        ctx = rng.integers(0, 4 * w + 1, n)
        g = engine.SharedGroups.find(t, ctx, 4)
        assert g.start[0] == 0 and g.start[-1] == n and (np.diff(g.start) > 0).all()
        for a, b in zip(g.start[:-1], g.start[1:]):
            p = int(g.prefix[a])
            assert (g.prefix[a:b] == p).all() and p % 4 == 0 and (ctx[a:b] >= p).all()
            assert (t[a:b, :p // 4] == t[a, :p // 4]).all()
            if b - a == 1:
                assert p == 0


# -- the engine ------------------------------------------------------------------------------

def test_caches_refuse_windows_that_do_not_fit(monkeypatch):
    make = lambda dt=torch.float16, **kw: engine.PagedKVCache(4, 2, 64, 16, dt, "cpu", 4, **kw)  # noqa: E731
    make(window=1)
    make(window=5, sinks=2)
    for kw in (dict(window=0), dict(window=-4), dict(window=4, sinks=-1), dict(sinks=3), dict(dt=torch.float8_e4m3fn, window=4)):
        with pytest.raises(ValueError):
            make(**kw)


def test_shared_steps_are_for_plain_16_bit_caches():
    for kw in (dict(dt=torch.float8_e4m3fn), dict(dt=torch.float16, window=8)):
        dt = kw.pop("dt")
        eng = engine.PagedKVCache(8, 2, 64, 16, dt, "cpu", 4, **kw)
        a = eng.new_sequence(20)
        plan = eng.plan_step([a, eng.fork(a)])
        assert eng.upload(plan).groups is None
        with pytest.raises(ValueError):
            eng.upload(plan, shared=True)


def test_upload_finds_forks():
    eng = engine.PagedKVCache(30, 2, 64, 16, torch.float16, "cpu", 8)
    a = eng.new_sequence(40)
    plan = eng.plan_step([a, eng.fork(a), eng.new_sequence(5)])
    g = eng.upload(plan, shared=True).groups
    assert g.start.tolist() == [0, 2, 3] and g.prefix.tolist() == [32, 32, 0]
    assert (g.max_prefix_len, g.max_group_size, g.max_suffix_len) == (32, 2, 9)
    assert eng.upload(eng.plan_step([eng.new_sequence(40)]), shared=True).groups is None


def prepared(eng, monkeypatch, groups=None, **kw):
    monkeypatch.setattr(engine, "_check_step", lambda *a, **k: 0)
    q, k, v = _tokens()
    step = engine.DeviceStep(slots=torch.arange(3), pairs=torch.zeros(0, 2, dtype=torch.int32),
                             tables=torch.zeros(3, 4, dtype=torch.int32), context_lens=torch.ones(3, dtype=torch.int32),
                             max_context_len=60, groups=groups)
    return eng.prepare(q, k, v, step, torch.zeros_like(q), scale=0.5, stream=STREAM, **kw), q, step


def test_a_prepared_step_with_a_window(world, monkeypatch):  # noqa: F811
    eng = engine.PagedKVCache(4, 2, 64, 16, torch.float16, "cpu", 4, window=7, sinks=2)
    step, q, dev = prepared(eng, monkeypatch)
    step()
    names = [n for n, _ in world.lib.calls if not n.startswith("pkv_")]
    assert names == ["kv_reshape_and_cache", "paged_attention_decode_window"]
    args = world.lib.calls[-1][1]
    assert args[6:18] == (3, 4, 60, 16, 4, 4, 2, 64, 0.5, 7, 2, 0) and args[18].value == 77
    with pytest.raises(ValueError):
        step.write_attend()
    with pytest.raises(ValueError):
        prepared(eng, monkeypatch, partition_size=64)


def test_a_prepared_step_with_groups(world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(engine, "paged_attention_decode_shared_workspace_size", lambda *a: 4096)
    eng = engine.PagedKVCache(4, 2, 64, 16, torch.float16, "cpu", 4)
    g = engine.DeviceGroups(torch.tensor([0, 2, 3], dtype=torch.int32), torch.tensor([16, 16, 0], dtype=torch.int32), 16, 2, 44)
    step, q, dev = prepared(eng, monkeypatch, groups=g)
    step()
    names = [n for n, _ in world.lib.calls if not n.startswith("pkv_")]
    assert names == ["kv_reshape_and_cache", "paged_attention_decode_shared"]
    args = world.lib.calls[-1][1]
    assert args[6:8] == (g.start.data_ptr(), g.prefix.data_ptr())
    assert args[8:21] == (3, 2, 2, 16, 44, 4, 60, 16, 4, 4, 2, 64, 0.5) and args[22] == 4096
    assert ((4096,), STREAM) in world.made               # the step's own memory, made on its stream
    with pytest.raises(ValueError):
        step.write_attend()


@pytest.fixture
def scratch(monkeypatch):
    """The binding's scratch with streams, captures and devices stood in for: state["capturing"], state["stream"]."""
    state = dict(capturing=False, stream=5)
    make = torch.empty
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_raw_stream", lambda s, index: s.cuda_stream if s else state["stream"])
    monkeypatch.setattr(pkv, "_capturing", lambda s: state["capturing"])
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state["capturing"], raising=False)
    monkeypatch.setattr(pkv, "_on", lambda s: __import__("contextlib").nullcontext())
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: make(*a, **kw))
    monkeypatch.setattr(pkv, "_scratches", __import__("threading").local())
    return state


def test_scratch_is_kept_per_stream_and_thread(scratch):
    a = pkv._scratch(0, 100, None)
    assert pkv._scratch(0, 50, None) is a and pkv._scratch(0, a.numel(), None) is a
    scratch["stream"] = 6
    b = pkv._scratch(0, 100, None)
    assert b is not a and pkv._scratch(0, 100, STREAM) is not b
    big = pkv._scratch(0, b.numel() + 1, None)
    assert big.numel() > b.numel() and pkv._scratch(0, 100, None) is big
    import threading
    got = []
    t = threading.Thread(target=lambda: got.append(pkv._scratch(0, 100, None)))
    t.start()
    t.join()
    assert got[0] is not big


def test_captured_calls_take_scratch_of_their_own(scratch):
    a = pkv._scratch(0, 100, None)
    scratch["capturing"] = True
    b, c = pkv._scratch(0, 100, None), pkv._scratch(0, 100, None)
    assert a is not b and b is not c
    scratch["capturing"] = False
    assert pkv._scratch(0, 100, None) is a
