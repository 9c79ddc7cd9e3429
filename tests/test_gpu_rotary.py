"""The rotary table and the rotating cache writes on the GPU, against the
formula on the CPU."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import F8, RefCache8, rotate32

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _theta(rot, base, scaling, factor, orig, low, high):
    i = np.arange(rot // 2, dtype=np.float64)
    w = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return w / factor
    if scaling == "by_parts":
        y = np.clip((orig * w / (2 * math.pi) - low) / (high - low), 0, 1)
        return w * (y + (1 - y) / factor)
    return w


@pytest.mark.parametrize("n,rot,base,scaling,factor,orig", [
    (1, 16, 1e4, "none", 1.0, 0), (257, 32, 1e4, "linear", 4.0, 0), (4097, 128, 5e5, "by_parts", 8.0, 512),
    (70001, 96, 1e4, "none", 1.0, 0), (131072, 64, 1e6, "by_parts", 5.5, 8192), (33, 256, 1.5, "none", 1.0, 0),
    (1000, 48, 1e4, "none", 1.0, 0),
])
@pytest.mark.parametrize("magnitude", [1.0, -0.75, 1.2079])
def test_table(cuda_device, n, rot, base, scaling, factor, orig, magnitude):
    """Off by: the turn's truncation (2 pi 2^-32), its remainder's conversion to fp32 and to an angle (2 pi / 4 *
    2^-24), the series' rounding (a step, 2^-24 below 1) and the magnitude's product and own rounding (2 * 2^-24):
    under 2^-22."""
    t = pkv.rotary_table(n, rot, base=base, scaling=scaling, factor=factor, original_positions=orig,
                         magnitude=magnitude, device=cuda_device).double().cpu().numpy()
    pkv.check()
    a = np.arange(n, dtype=np.float64)[:, None] * _theta(rot, base, scaling, factor, orig, 1.0, 32.0)
    want = magnitude * np.stack([np.cos(a), np.sin(a)], -1)
    assert np.abs(t - want).max() <= 2.0 ** -22 * max(1.0, abs(magnitude))


def test_table_writes_nothing_behind(cuda_device):
    buf = torch.full((40, 24, 2), 7.0, device=cuda_device)
    pkv.rotary_table(33, 48, out=buf[:33])
    assert bool((buf[33:] == 7.0).all()) and bool((buf[:33, 0].square().sum(-1) - 1 < 1e-6).all())


class Inputs:
    def __init__(self, dev, T, H, Hkv, d, B, dtype, seed, rot, pad=0.2, NB=None, strided=True, maxpos=777):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.NB = NB or (T // B + 9)
        dt = DT[dtype]
        qkv = torch.randn(T, H + 2 * Hkv + 1, d, generator=g).to(dt)
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:H + 2 * Hkv]
        if not strided:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
            self.dq, self.dk, self.dv = (x.to(dev) for x in (self.q, self.k, self.v))
        else:
            dq = qkv.to(dev)
            self.dq, self.dk, self.dv = dq[:, :H], dq[:, H:H + Hkv], dq[:, H + Hkv:H + 2 * Hkv]
        self.positions = rng.integers(0, maxpos, T).astype(np.int32)
        self.slots = rng.choice(self.NB * B, T, replace=False).astype(np.int64)
        self.slots[rng.random(T) < pad] = -1
        i = np.arange(rot // 2)
        a = np.arange(maxpos)[:, None] * 10000.0 ** (-2.0 * i / max(rot, 1))
        self.cs = torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1)).float()
        self.dpos, self.dslots, self.dcs = (torch.as_tensor(x).to(dev) for x in (self.positions, self.slots, self.cs))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("T,H,Hkv,B", [(1, 4, 4, 16), (37, 7, 1, 4), (130, 8, 2, 128)])
def test_append_is_the_formula(cuda_device, layout, dtype, d, rot, T, H, Hkv, B):
    x = Inputs(cuda_device, T, H, Hkv, d, B, dtype, T * 100 + rot, rot, strided=T != 37)
    dt = DT[dtype]
    kc0, vc0 = torch.randn(x.NB, Hkv, B, d).to(dt), torch.randn(x.NB, Hkv, B, d).to(dt)
    kc, vc = kc0.to(cuda_device), vc0.to(cuda_device)
    q = pkv.kv_rotary_and_cache(x.dq, x.dk, x.dv, x.dcs, x.dpos, kc, vc, x.dslots, layout=layout)
    pkv.check()
    assert torch.equal(q.cpu(), rotate32(x.q, x.cs, x.positions, rot, layout).to(dt))
    k = rotate32(x.k, x.cs, x.positions, rot, layout).to(dt)
    for t, s in enumerate(x.slots):
        if s >= 0:
            kc0[s // B, :, s % B], vc0[s // B, :, s % B] = k[t], x.v[t]
    assert torch.equal(kc.cpu(), kc0) and torch.equal(vc.cpu(), vc0)


def test_append_in_place_without_queries_and_on_a_stream(cuda_device):
    x = Inputs(cuda_device, 50, 4, 2, 128, 16, "bf16", 3, 128, strided=False)
    kc, vc = (torch.zeros(x.NB, 2, 16, 128, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    want = rotate32(x.q, x.cs, x.positions, 128, "half").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = pkv.kv_rotary_and_cache(x.dq, x.dk, x.dv, x.dcs, x.dpos, kc, vc, x.dslots, query_out=x.dq, stream=s)
    s.synchronize()
    assert out.data_ptr() == x.dq.data_ptr() and torch.equal(x.dq.cpu(), want)
    assert pkv.kv_rotary_and_cache(None, x.dk, x.dv, x.dcs, x.dpos, k2, v2, x.dslots) is None
    pkv.check()
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_positions_and_slots_are_latched(cuda_device, fp8):
    B, Hkv, d = 16, 2, 64
    x = Inputs(cuda_device, 6, 4, Hkv, d, B, "f16", 5, 64, pad=0.0, NB=8)
    dt = F8 if fp8 else torch.float16
    kc, vc = (torch.zeros(8, Hkv, B, d, device=cuda_device).to(dt) for _ in range(2))
    sc = pkv.kv_scales(8, Hkv, cuda_device)

    def call(slots, positions):
        args = (x.dq, x.dk, x.dv, x.dcs, torch.tensor(positions, dtype=torch.int32, device=cuda_device), kc, vc)
        slots = torch.tensor(slots, device=cuda_device)
        if fp8:
            pkv.kv_rotary_and_cache_fp8(*args, sc, slots)
        else:
            pkv.kv_rotary_and_cache(*args, slots)

    ok = [0, 16, 32, 48, 64, 80]
    for slots, positions, word in ((ok, [0, 1, 777, 3, 4, 5], "position"), (ok, [0, -1, 2, 3, 4, 5], "position"),
                                   ([0, 16, 128, 48, 64, 80], [0] * 6, "slot")):
        call(slots, positions)
        with pytest.raises(pkv.PkvError) as e:
            pkv.check()
        assert e.value.status_name == "PKV_EINDEX" and word in str(e.value)
    # a padding token may carry any position
    call([0, -1, 32, 48, 64, 80], [0, -5, 2, 3, 4, 5])
    pkv.check()


def _random_cache8(NB, Hkv, B, d, seed):
    rng = np.random.default_rng(seed)
    codes = [torch.from_numpy(rng.integers(0, 256, (NB, Hkv, B, d)).astype(np.uint8)) for _ in range(2)]
    codes = [torch.where((c & 0x7F) == 0x7F, c & 0xF0, c) for c in codes]
    sc = torch.from_numpy((2.0 ** rng.integers(-12, 3, (NB, Hkv + Hkv % 2, 2))).astype(np.float32))
    return codes[0].view(F8), codes[1].view(F8), sc


def _runs(rng, NB, B, T):
    """Slots sequence by sequence: some from a block's start, some into a partly filled block, some across blocks."""
    order = list(rng.permutation(NB))
    slots = []
    while len(slots) < T:
        b = order.pop()
        lo = int(rng.integers(0, B)) if rng.random() < 0.6 else 0
        hi = int(rng.integers(lo + 1, B + 1)) if rng.random() < 0.5 else B
        slots += [b * B + o for o in range(lo, hi)]
        if rng.random() < 0.3:
            slots += [-1]
    return np.array(slots[:T], np.int64)


def _same8(ref, kc, vc, sc, what):
    for i, c in enumerate((kc, vc)):
        got = c.cpu().view(torch.uint8).numpy()
        nan = (got & 0x7F) == 0x7F
        assert np.array_equal(nan, (ref.codes[i] & 0x7F) == 0x7F), what
        assert np.array_equal(got[~nan], ref.codes[i][~nan]), what
    assert np.array_equal(sc.cpu().numpy(), ref.scales), what


@pytest.mark.parametrize("B", [4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("d,rot,layout", [(64, 32, "half"), (128, 128, "half"), (128, 64, "interleaved"), (64, 0, "half")])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append8_is_the_definition(cuda_device, B, d, rot, layout, dtype):
    """Several calls on one cache, the later ones larger: scales grow and the blocks' other rows are rounded again."""
    Hkv, H = 3, 6
    rng = np.random.default_rng(B + d)
    NB = 40
    k0, v0, s0 = _random_cache8(NB, Hkv, B, d, B)
    kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
    ref = RefCache8(k0, v0, s0)
    for call, T in enumerate((1, 5 * B // 2 + 3, 33, 9 * B)):
        x = Inputs(cuda_device, T, H, Hkv, d, B, dtype, call, rot, NB=NB, strided=call % 2 == 0)
        grow = 2.0 ** (3 * call - 4)
        x.k, x.dk, x.v, x.dv = x.k * grow, x.dk * grow, x.v * grow, x.dv * grow
        slots = _runs(rng, NB, B, T)
        dslots = torch.from_numpy(slots).to(cuda_device)
        args = (x.dq, x.dk, x.dv, x.dcs, x.dpos) if rot else (None, x.dk, x.dv, None, None)
        q = pkv.kv_rotary_and_cache_fp8(*args, kc, vc, sc, dslots, layout=layout)
        pkv.check()
        if rot:
            assert torch.equal(q.cpu(), rotate32(x.q, x.cs, x.positions, rot, layout).to(DT[dtype]))
        ref.append(rotate32(x.k, x.cs, x.positions, rot, layout).numpy(), x.v.float().numpy(), slots)
        _same8(ref, kc, vc, sc, f"call {call}")


def test_append8_long_call(cuda_device):
    """Enough tokens that a CTA looks over several."""
    T, B, Hkv, d = 12001, 16, 1, 64
    x = Inputs(cuda_device, T, 2, Hkv, d, B, "f16", 1, 64, NB=900)
    order = np.random.default_rng(2).permutation(900)
    slots = np.concatenate([b * B + np.arange(B) for b in order])[3:T + 3].astype(np.int64)
    k0, v0, s0 = _random_cache8(900, Hkv, B, d, 7)
    kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
    pkv.kv_rotary_and_cache_fp8(x.dq, x.dk, x.dv, x.dcs, x.dpos, kc, vc, sc, torch.from_numpy(slots).to(cuda_device))
    pkv.check()
    ref = RefCache8(k0, v0, s0)
    ref.append(rotate32(x.k, x.cs, x.positions, 64, "half").numpy(), x.v.float().numpy(), slots)
    _same8(ref, kc, vc, sc, "long")


@pytest.mark.parametrize("T,Hkv", [(1023, 1), (1024, 3), (1500, 40)])
def test_append8_large_step(cuda_device, T, Hkv):
    """One token for each of many sequences, some padded, some blocks begun anew, scales that grow; a few runs of two."""
    B, d, NB = 16, 64, 1600
    x = Inputs(cuda_device, T, 2, Hkv, d, B, "bf16", 3, 32, NB=NB)
    rng = np.random.default_rng(4)
    x.k, x.dk = x.k * 8, x.dk * 8
    for pairs in (False, True):
        slots = rng.permutation(NB)[:T].astype(np.int64) * B + rng.integers(0, B - 1, T)
        slots[rng.random(T) < 0.1] = -1
        if pairs:
            slots[701], slots[31] = slots[700] + 1, slots[30] + 1
            slots[700] = -1 if slots[700] < 0 else slots[700]
            slots[[31, 701]] = np.where(slots[[30, 700]] < 0, -1, slots[[31, 701]])
        k0, v0, s0 = _random_cache8(NB, Hkv, B, d, 8)
        kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
        q = pkv.kv_rotary_and_cache_fp8(x.dq, x.dk, x.dv, x.dcs, x.dpos, kc, vc, sc, torch.from_numpy(slots).to(cuda_device))
        pkv.check()
        assert torch.equal(q.cpu(), rotate32(x.q, x.cs, x.positions, 32, "half").bfloat16())
        ref = RefCache8(k0, v0, s0)
        ref.append(rotate32(x.k, x.cs, x.positions, 32, "half").numpy(), x.v.float().numpy(), slots)
        _same8(ref, kc, vc, sc, "step")


@pytest.mark.parametrize("T,H,Hkv,B,d", [(5, 2, 2, 128, 128), (40, 8, 8, 16, 128), (200, 2, 40, 16, 64), (300, 7, 1, 4, 64),
                                         (700, 4, 2, 32, 128), (2100, 6, 3, 16, 64), (9000, 2, 1, 8, 64)])
def test_append8_short_runs(cuda_device, T, H, Hkv, B, d):
    """A few tokens for each of many sequences, runs of one among them, padding between."""
    x = Inputs(cuda_device, T, H, Hkv, d, B, "f16", T, d, NB=T + 8)
    x.k, x.dk = x.k * 4, x.dk * 4
    rng = np.random.default_rng(T)
    slots, free = [], list(rng.permutation(T + 8))
    while len(slots) < T:
        n = int(rng.integers(1, min(6, B + 1)))
        lo = 0 if rng.random() < 0.3 else int(rng.integers(0, B - n + 1))
        slots += list(free.pop() * B + lo + np.arange(n)) + [-1] * int(rng.random() < 0.1)
    slots = np.array(slots[:T], np.int64)
    k0, v0, s0 = _random_cache8(T + 8, Hkv, B, d, 9)
    kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
    q = pkv.kv_rotary_and_cache_fp8(x.dq, x.dk, x.dv, x.dcs, x.dpos, kc, vc, sc, torch.from_numpy(slots).to(cuda_device))
    pkv.check()
    assert torch.equal(q.cpu(), rotate32(x.q, x.cs, x.positions, d, "half").half())
    ref = RefCache8(k0, v0, s0)
    ref.append(rotate32(x.k, x.cs, x.positions, d, "half").numpy(), x.v.float().numpy(), slots)
    _same8(ref, kc, vc, sc, "short runs")


def test_append8_special_values(cuda_device):
    """Zeros, the least and the largest magnitudes, infinities and NaN: what the definition says of each."""
    B, d = 8, 64
    for dtype, top, tiny in ((torch.float16, 65504.0, 2.0 ** -24), (torch.bfloat16, 3.3895e38, 2.0 ** -133)):
        rows = torch.zeros(8, 1, d)
        rows[1] = tiny
        rows[2, 0, 0], rows[2, 0, 1] = top, -top
        rows[3, 0, 0] = math.inf
        rows[4, 0, 0] = math.nan
        rows[4, 0, 1] = 3.0
        rows[5, 0, 0] = 448.0
        rows[6, 0, 0] = 450.0
        rows[7, 0, :16] = torch.linspace(-1, 1, 16)
        k = rows.to(dtype)
        slots = np.arange(8, dtype=np.int64) * B          # a block each, started anew
        k0, v0, s0 = _random_cache8(8, 1, B, d, 3)
        s0[:] = math.nan                                    # what a fresh block held does not matter
        kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
        dk = k.to(cuda_device)
        pkv.kv_rotary_and_cache_fp8(None, dk, dk, None, None, kc, vc, sc, torch.from_numpy(slots).to(cuda_device))
        pkv.check()
        ref = RefCache8(k0, v0, s0)
        ref.append(k.float().numpy(), k.float().numpy(), slots)
        got, want = sc.cpu().numpy()[:, :1], ref.scales[:, :1]
        assert np.array_equal(got, want)
        for i, c in enumerate((kc, vc)):
            g = c.cpu().view(torch.uint8).numpy()
            nan = (g & 0x7F) == 0x7F
            assert np.array_equal(nan, (ref.codes[i] & 0x7F) == 0x7F)
            assert np.array_equal(g[~nan], ref.codes[i][~nan])


def test_append_empty_launches_nothing(cuda_device):
    kc = torch.zeros(2, 1, 16, 64, dtype=F8, device=cuda_device)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=cuda_device)
    before = pkv.launch_count()
    pkv.kv_rotary_and_cache_fp8(None, e, e, None, None, kc, kc.clone(), pkv.kv_scales(2, 1, cuda_device),
                                torch.empty(0, dtype=torch.int64, device=cuda_device))
    assert pkv.launch_count() == before
