"""Argument checks of the rotary and 8-bit calls (CPU: nothing is launched),
and what the tests' own 8-bit reference rests on."""
import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import e4m3_values, pow2_scale, rotate32, to_code
from paged_kv_cache_139_gb300 import _lib

P = 16          # an aligned address that nothing reads


def _message():
    return _lib.load().pkv_last_error_string().decode()


def _call(name, order, defaults, over):
    args = dict(defaults, **over)
    rc = getattr(_lib.load(), name)(*(args[k] for k in order))
    return rc


TABLE = dict(out=P, n=10, rot=64, base=1e4, scaling=0, factor=1.0, orig=0, low=1.0, high=32.0, mag=1.0, st=None)


@pytest.mark.parametrize("over", [
    dict(out=None), dict(out=24), dict(n=-1), dict(rot=0), dict(rot=24), dict(rot=272), dict(base=1.0),
    dict(base=float("nan")), dict(base=float("inf")), dict(mag=float("nan")), dict(scaling=3), dict(scaling=1, factor=0.5),
    dict(scaling=1, factor=float("inf")), dict(scaling=2, factor=2.0), dict(scaling=2, factor=2.0, orig=100, low=4.0, high=4.0),
])
def test_table_refusals(over):
    assert _call("rotary_table", TABLE, TABLE, over) == 1 and "rotary_table" in _message()


@pytest.mark.parametrize("over", [dict(n=2 ** 30 + 1), dict(n=2 ** 31 - 1), dict(mag=1e39), dict(mag=-float("inf"))])
def test_table_limits(over):
    """Positions past the end of the table's stretches have to fit 31 bits, the magnitude fp32."""
    assert _call("rotary_table", TABLE, TABLE, over) == 1 and "rotary_table" in _message()


def test_empty_calls_are_ok():
    assert _call("rotary_table", TABLE, TABLE, dict(n=0)) == 0
    assert _append(False, T=0) == 0 and _append(True, T=0) == 0
    assert _decode(S=0) == 0 and _prefill(S=0) == 0 and _prefill(T=0) == 0


APPEND = dict(qo=P, q=P, k=P, v=P, kc=P, vc=P, sc=P, cs=P, pos=P, slots=P, T=4, H=4, Hkv=2, d=128, rot=128, npos=10, layout=0,
              qs=512, ks=256, vs=256, B=16, NB=8, dt=0, st=None)


def _append(fp8, **over):
    order = [k for k in APPEND if fp8 or k != "sc"]
    return _call("kv_rotary_and_cache_fp8" if fp8 else "kv_rotary_and_cache", order, APPEND, over)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over", [
    dict(T=-1), dict(H=-1), dict(Hkv=0), dict(d=96), dict(d=256), dict(rot=8), dict(rot=144), dict(rot=-16), dict(npos=-1),
    dict(layout=2), dict(qs=504), dict(qs=516), dict(ks=248), dict(ks=257), dict(vs=0), dict(B=12), dict(B=0), dict(NB=-1),
    dict(dt=2), dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(cs=None),
    dict(pos=None), dict(slots=None), dict(q=24), dict(kc=8), dict(cs=4), dict(T=2 ** 31 - 1, H=65536, qs=2 ** 24),
])
def test_append_refusals(fp8, over):
    assert _append(fp8, **over) == 1 and "kv_rotary_and_cache" in _message()


@pytest.mark.parametrize("over", [dict(sc=None), dict(sc=8), dict(B=256), dict(B=2), dict(rot=0, cs=None, pos=None)])
def test_append8_refusals(over):
    """Also: queries with nothing to rotate them by."""
    assert _append(True, **over) == 1


def test_append_needs_a_rotation():
    assert _append(False, rot=0) == 1


DECODE = dict(out=P, q=P, kc=P, vc=P, sc=P, bt=P, cl=P, S=2, mb=4, mcl=0, B=16, NB=8, H=4, Hkv=2, d=128, scale=0.1, part=0, ws=P,
              wsb=1 << 30, dt=0, st=None)


def _decode(**over):
    return _call("paged_attention_decode_fp8", DECODE, DECODE, over)


@pytest.mark.parametrize("over", [
    dict(d=96), dict(d=256), dict(B=12), dict(B=2), dict(B=256), dict(H=5), dict(H=0), dict(Hkv=0), dict(part=32), dict(part=-64),
    dict(mcl=65), dict(mcl=-1), dict(dt=2), dict(S=-1), dict(S=65536), dict(NB=-1), dict(mb=-1), dict(out=None), dict(q=None),
    dict(kc=None), dict(sc=None), dict(bt=None), dict(cl=None), dict(q=18), dict(sc=8), dict(ws=None), dict(ws=24), dict(wsb=128),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(mb=1 << 24, part=64), dict(H=65536),
])
def test_decode_refusals(over):
    assert _decode(**over) == 1 and "paged_attention_decode_fp8" in _message()


PREFILL = dict(out=P, q=P, kc=P, vc=P, sc=P, bt=P, cl=P, qst=P, S=2, T=10, mql=0, mcl=0, mb=4, B=16, NB=8, H=4, Hkv=2, d=128,
               scale=0.1, ws=P, wsb=1 << 30, dt=0, st=None)


def _prefill(**over):
    return _call("paged_attention_prefill_fp8", PREFILL, PREFILL, over)


@pytest.mark.parametrize("over", [
    dict(d=96), dict(B=12), dict(B=2), dict(B=256), dict(H=5), dict(Hkv=0), dict(dt=2), dict(S=-1), dict(S=65536), dict(T=-1),
    dict(mql=-1), dict(mcl=-1), dict(mcl=65), dict(mb=0), dict(mb=-1), dict(mb=1 << 28), dict(NB=0), dict(NB=-1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(qst=None), dict(sc=None),
    dict(kc=18), dict(ws=None), dict(ws=24), dict(wsb=128),
])
def test_prefill_refusals(over):
    assert _prefill(**over) == 1


def test_workspace_sizes():
    size = pkv.paged_attention_decode_fp8_workspace_size
    head = 256
    assert size(2, 4, 2, 128, 64, 64) == head == size(2, 4, 2, 128, 0, 0)
    r = lambda x: (x + 255) // 256 * 256  # noqa: E731
    n = 8 * 32 * (32768 // 512)
    assert size(8, 32, 8, 128, 32768, 512) == head + 2 * r(4 * n) + r(4 * n * 128)
    blocks = 3 * 7
    assert pkv.paged_attention_prefill_fp8_workspace_size(3, 2, 64, 16, 100) == head + r(4 * blocks) + 2 * r(
        blocks * 2 * 16 * 64 * 2)
    L = _lib.load()
    assert L.paged_attention_fp8_workspace_init(None, 1 << 20, None) == 1
    assert L.paged_attention_fp8_workspace_init(P, head - 16, None) == 1
    assert L.paged_attention_fp8_workspace_init(24, 1 << 20, None) == 1


def test_scales_shape():
    assert pkv.kv_scales(5, 3, "cpu").shape == (5, 4, 2) and pkv.kv_scales(5, 8, "cpu").shape == (5, 8, 2)


# -- the reference -------------------------------------------------------------------

def test_reference_codes_are_the_formats():
    v = e4m3_values()
    t = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    x = (torch.randn(50000) * torch.randn(50000).mul(4).exp()).clamp(-448, 448)
    x = torch.cat([x, torch.from_numpy(np.concatenate([v[~np.isnan(v)], (v[:125] + v[1:126]) / 2])).float()])
    assert np.array_equal(to_code(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scale_is_the_least():
    for a in (1e-30, 0.3, 1.75, 1.7500001, 448.0, 449.0, 896.0, 65504.0, 3e38):
        s = pow2_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -60 or a > 224 * s)


def test_reference_rotation_turns_pairs():
    """Rotating by p then reading the dot product depends on the distance of two positions only."""
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn(1, 1, 64, generator=g).double(), torch.randn(1, 1, 64, generator=g).double()
    a = torch.arange(50).double()[:, None] * 10000.0 ** (-2.0 * torch.arange(32) / 64)
    cs = torch.stack([a.cos(), a.sin()], -1).float()
    for layout in ("half", "interleaved"):
        dots = [float((rotate32(q, cs, [p + 7], 64, layout) * rotate32(k, cs, [p], 64, layout)).sum()) for p in (0, 11, 42)]
        assert max(dots) - min(dots) < 1e-4
        assert torch.equal(rotate32(q, cs, [0], 64, layout), q.float())


def test_plan_positions():
    from paged_kv_cache_139_gb300.engine import PrefillPlan, StepPlan
    e = np.empty((0, 2), np.int32)
    ctx = np.array([5, 1, 40], np.int32)
    assert StepPlan(np.arange(3), np.zeros(3, np.int64), e, e, ctx).positions.tolist() == [4, 0, 39]
    p = PrefillPlan(np.arange(4), np.zeros(9, np.int64), e, e, np.array([5, 7, 40, 3], np.int32),
                    np.array([0, 5, 5, 8, 9], np.int32))
    assert p.positions.tolist() == [0, 1, 2, 3, 4, 37, 38, 39, 2] and p.positions.dtype == np.int32
