"""The engine over a cache with rotary positions, in 8 and in 16 bits: prompts,
a fork, decode steps with copy-on-write, swapping out and in, checked step by
step against the definitions on the CPU (the 8-bit cache code by code)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import F8, RefCache8, attention64, attention_tolerance, rotate32
from paged_kv_cache_139_gb300.engine import HostKVPool, PagedKVCache, RotaryPositions

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Ref16:
    def __init__(self, NB, Hkv, B, d, dtype):
        self.pools = [torch.zeros(NB, Hkv, B, d, dtype=dtype) for _ in range(2)]
        self.B = B

    def append(self, k32, v32, slots):
        for t, s in enumerate(slots):
            for pool, x in zip(self.pools, (k32, v32)):
                pool[s // self.B, :, s % self.B] = torch.as_tensor(x[t]).to(pool.dtype)

    def copy(self, pairs):
        for pool in self.pools:
            for src, dst in pairs:
                pool[dst] = pool[src].clone()

    def values(self, i):
        return self.pools[i].double().numpy()


class Ref8(RefCache8):
    def copy(self, pairs):
        for pool in (*self.codes, self.scales):
            for src, dst in pairs:
                pool[dst] = pool[src].copy()


class World:
    def __init__(self, dev, fp8, dtype, H, Hkv, d, B, layout, rot):
        self.dev, self.dtype, self.H, self.Hkv, self.d, self.B = dev, DT[dtype], H, Hkv, d, B
        self.g = torch.Generator().manual_seed(d + B)
        NB = 96
        self.rotary = RotaryPositions.make(2048, rot, dev, layout=layout, scaling="by_parts", factor=4.0,
                                           original_positions=512) if rot else None
        cs = self.rotary.cos_sin.cpu() if rot else None
        self.turn = (lambda x, pos: rotate32(x, cs, pos, rot, layout)) if rot else (lambda x, pos: x.float())
        order = np.random.default_rng(B).permutation(NB)
        self.eng = PagedKVCache(NB, Hkv, d, B, F8 if fp8 else self.dtype, dev, 64, order, rotary=self.rotary)
        for pool in self.eng._pools():
            pool.zero_()
        self.ref = Ref8(self.eng.key_cache, self.eng.value_cache, self.eng.scales) if fp8 else Ref16(NB, Hkv, B, d, self.dtype)
        self.fp8 = fp8
        self.decode_bits, self.prefill_bits = (21 if fp8 else (10 if dtype == "f16" else 7)), (10 if dtype == "f16" else 14)

    def tokens(self, T, grow):
        x = [torch.randn(T, h, self.d, generator=self.g) for h in (self.H, self.Hkv, self.Hkv)]
        return x[0].to(self.dtype), (x[1] * grow).to(self.dtype), (x[2] * grow).to(self.dtype)

    def expect(self, out, q, plan, starts, bits):
        eps = torch.finfo(self.dtype).eps
        k, v = self.ref.values(0), self.ref.values(1)
        for s, n in enumerate(plan.context_lens):
            rows = slice(int(starts[s]), int(starts[s + 1]))
            want, mag, vmax = attention64(q[rows].double().numpy(), k, v, plan.tables[s], int(n), 1 / math.sqrt(self.d))
            tol = attention_tolerance(want, mag, vmax, int(n), self.d, eps, bits)
            got = out[rows].double().cpu().numpy()
            assert np.all(np.abs(got - want) <= tol), (s, np.abs(got - want).max(), tol.min())

    def same_cache(self):
        if self.fp8:
            for pool, codes in zip((self.eng.key_cache, self.eng.value_cache), self.ref.codes):
                assert np.array_equal(pool.view(torch.uint8).cpu().numpy(), codes)
            assert np.array_equal(self.eng.scales.cpu().numpy(), self.ref.scales)
        else:
            for pool, want in zip((self.eng.key_cache, self.eng.value_cache), self.ref.pools):
                assert torch.equal(pool.cpu(), want)

    def write_ref(self, plan, q, k, v):
        pos = plan.positions
        self.ref.copy(plan.pairs)
        self.ref.append(self.turn(k, pos).numpy(), v.float().numpy(), plan.slots)
        return self.turn(q, pos).to(self.dtype)

    def prompt(self, seqs, new, prepared):
        plan = self.eng.plan_prefill(seqs, new)
        step = self.eng.upload_prefill(plan)
        q, k, v = self.tokens(sum(new), 1.0)
        dq, dk, dv = (x.to(self.dev) for x in (q, k, v))
        if prepared:
            out = torch.empty_like(dq)
            self.eng.prepare_prefill(dq, dk, dv, step, out)()
        else:
            out = self.eng.prefill(dq, dk, dv, step)
        pkv.check()
        self.expect(out, self.write_ref(plan, q, k, v), plan, plan.query_start, self.prefill_bits)
        self.same_cache()

    def step(self, seqs, grow, prepared):
        plan = self.eng.plan_step(seqs)
        step = self.eng.upload(plan)
        q, k, v = self.tokens(len(seqs), grow)
        dq, dk, dv = (x.to(self.dev) for x in (q, k, v))
        if prepared:
            out = torch.empty_like(dq)
            self.eng.prepare(dq, dk, dv, step, out)()
        else:
            out = self.eng.decode(dq, dk, dv, step)
        pkv.check()
        self.expect(out, self.write_ref(plan, q, k, v), plan, np.arange(len(seqs) + 1), self.decode_bits)
        self.same_cache()


@pytest.mark.parametrize("fp8,dtype,H,Hkv,d,B,layout,rot", [
    (True, "bf16", 8, 2, 128, 16, "half", 128), (True, "f16", 6, 3, 64, 8, "interleaved", 32), (True, "f16", 2, 2, 64, 32, "half", 0),
    (False, "bf16", 8, 2, 128, 16, "interleaved", 64), (False, "f16", 2, 2, 64, 4, "half", 64)])
def test_a_conversation(cuda_device, fp8, dtype, H, Hkv, d, B, layout, rot):
    w = World(cuda_device, fp8, dtype, H, Hkv, d, B, layout, rot)
    a, b = w.eng.new_sequence(0), w.eng.new_sequence(0)
    w.prompt([a, b], [37, 20], prepared=False)
    c = w.eng.fork(a)                                      # shares a's partly filled last block
    for i in range(4):
        w.step([a, b, c], 1.0 + 3.0 * (i == 2), prepared=i % 2 == 1)     # the third token is large: scales grow
    w.prompt([b], [45], prepared=True)                     # a second turn of b's
    host = HostKVPool(40, Hkv, d, B, F8 if fp8 else DT[dtype])
    ids, out_pairs = w.eng.swap_out([a, c], host)
    torch.cuda.synchronize()
    w.step([b], 1.0, prepared=False)
    (a2, c2), in_pairs = w.eng.swap_in(ids, host)
    torch.cuda.synchronize()
    # the blocks came back to other places: the reference moves them by way of the same host blocks
    back = {int(h): int(g) for h, g in in_pairs}
    held = {int(h): [np.array(p[int(g)]) if fp8 else p[int(g)].clone() for p in _ref_pools(w.ref)] for g, h in out_pairs}
    for h, pieces in held.items():
        for pool, piece in zip(_ref_pools(w.ref), pieces):
            pool[back[h]] = torch.as_tensor(piece) if not fp8 else piece
    w.step([a2, b, c2], 1.0, prepared=True)


def _ref_pools(ref):
    return (*ref.codes, ref.scales) if isinstance(ref, Ref8) else tuple(ref.pools)


def test_an_8_bit_cache_does_not_swap_with_a_16_bit_pool(cuda_device):
    eng = PagedKVCache(8, 2, 64, 16, F8, cuda_device, 4)
    s = eng.new_sequence(5)
    with pytest.raises(ValueError):
        eng.swap_out([s], HostKVPool(8, 2, 64, 16, torch.float16))
    assert eng.alloc.seq_len(s) == 5


def test_a_captured_step_replays(cuda_device):
    """The prepared calls of a step (rotating 8-bit write, attention) captured once and replayed over changing inputs and
    lengths give what the eager calls give."""
    H, Hkv, d, B, S = 8, 2, 64, 16, 5
    rotary = RotaryPositions.make(512, 64, cuda_device)
    engines = [PagedKVCache(80, Hkv, d, B, F8, cuda_device, 16, rotary=rotary) for _ in range(2)]
    for e in engines:
        for pool in e._pools():
            pool.zero_()
    seqs = [[e.new_sequence(0) for _ in range(S)] for e in engines]
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.empty(S, h, d, dtype=torch.bfloat16, device=cuda_device) for h in (H, Hkv, Hkv))
    out = [torch.empty_like(q) for _ in engines]
    fixed = graph = None
    for i in range(40):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g) * (1 + i % 3))
        steps = [e.upload(e.plan_step(s)) for e, s in zip(engines, seqs)]
        engines[0].prepare(q, k, v, steps[0], out[0])()
        if graph is None:
            fixed = steps[1]
            fixed.max_context_len = 256
            stream = torch.cuda.Stream()
            prep = engines[1].prepare(q, k, v, fixed, out[1], stream=stream)
            torch.cuda.synchronize()
            prep()                                   # kernels are set up outside capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                prep()
        else:
            for name in ("slots", "tables", "context_lens", "positions"):
                getattr(fixed, name).copy_(getattr(steps[1], name))
            graph.replay()
        torch.cuda.synchronize()
        pkv.check()
        for a, b in zip(engines[0]._pools(), engines[1]._pools()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        # another partition size (the captured call's bound is larger) sums in another order
        assert torch.allclose(out[0].float(), out[1].float(), rtol=2.0 ** -7, atol=2.0 ** -12 * float(v.abs().max()))


def test_bindings_refuse_what_does_not_fit(cuda_device):
    dev = cuda_device
    kc = torch.zeros(4, 2, 16, 64, dtype=F8, device=dev)
    sc = pkv.kv_scales(4, 2, dev)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device=dev)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=dev)
    cs = pkv.rotary_table(32, 64, device=dev)
    pos = torch.zeros(3, dtype=torch.int32, device=dev)
    slots = torch.arange(3, device=dev)
    call = lambda **o: pkv.kv_rotary_and_cache_fp8(*(dict(dict(q=q, k=k, v=k, cs=cs, pos=pos, kc=kc, vc=kc.clone(), sc=sc, s=slots), **o)[n]  # noqa: E731
                                                     for n in ("q", "k", "v", "cs", "pos", "kc", "vc", "sc", "s")))
    call()
    for o in (dict(k=k.bfloat16()), dict(v=k.float()), dict(q=q.cpu()), dict(kc=kc.view(torch.uint8)), dict(pos=pos.long()),
              dict(s=slots.int()), dict(sc=sc.double()), dict(k=k.float(), v=k.float(), q=q.float())):
        with pytest.raises(TypeError):
            call(**o)
    for o in (dict(k=k[:, :1]), dict(k=k[:, :, ::2]), dict(v=k.expand(1, 3, 2, 64)[0].transpose(0, 1)), dict(pos=pos[:2]),
              dict(sc=sc[:, :1]), dict(s=slots[:2]), dict(cs=cs[..., 0]), dict(cs=None, pos=None), dict(k=k[:1].expand(3, 2, 64)),
              dict(pos=None)):
        with pytest.raises(ValueError):
            call(**o)
    with pytest.raises(ValueError):
        pkv.kv_rotary_and_cache_fp8(q, k, k, cs, pos, kc, kc.clone(), sc, slots, layout="pairs")
    with pytest.raises(pkv.PkvError):                      # a table wider than the head
        call(cs=pkv.rotary_table(32, 128, device=dev))
    with pytest.raises(ValueError):
        pkv.rotary_table(32, 64, scaling="ntk", device=dev)
    out = torch.empty_like(q)
    bt, cl = torch.zeros(3, 1, dtype=torch.int32, device=dev), torch.ones(3, dtype=torch.int32, device=dev)
    pkv.paged_attention_decode_fp8(out, q, kc, kc, sc, bt, cl)
    for o in (dict(out=out.bfloat16()), dict(q=q.float()), dict(kc=kc.half()), dict(bt=bt.long()), dict(cl=cl.cpu())):
        a = dict(dict(out=out, q=q, kc=kc, bt=bt, cl=cl), **o)
        with pytest.raises((TypeError, ValueError)):
            pkv.paged_attention_decode_fp8(a["out"], a["q"], a["kc"], kc, sc, a["bt"], a["cl"])
    pkv.check()
