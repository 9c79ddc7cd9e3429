"""The engine with a sliding window and with shared prefixes: prompts, forks and
decode steps (direct, prepared and captured), checked step by step against 64
bits on the CPU."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import rotate32
from paged_kv_cache_139_gb300.engine import GraphStep, PagedKVCache, RotaryPositions, StagedInputs
from span_reference import DT, attention64, check, visible

pytestmark = pytest.mark.gpu


class World:
    """An engine and, per sequence id, the keys and values it has been given (as they lie in the cache)."""

    def __init__(self, dev, dtype, H, Hkv, d, B, window=None, sinks=0, rot=0, NB=300):
        self.dev, self.dtype, self.H, self.Hkv, self.d = dev, dtype, H, Hkv, d
        self.rotary = RotaryPositions.make(4096, rot, dev) if rot else None
        self.rot = rot
        kw = dict(window=window, sinks=sinks) if window else {}
        self.eng = PagedKVCache(NB, Hkv, d, B, DT[dtype], dev, 128, np.random.default_rng(B).permutation(NB),
                                rotary=self.rotary, **kw)
        for pool in self.eng._pools():
            pool.fill_(math.nan)
        self.window, self.sinks = (window, sinks) if window else (1 << 40, 0)
        self.g = torch.Generator().manual_seed(H + d)
        self.kv = {}

    def tokens(self, T):
        return [torch.randn(T, h, self.d, generator=self.g).to(DT[self.dtype]) for h in (self.H, self.Hkv, self.Hkv)]

    def turn(self, x, pos):
        if not self.rot:
            return x
        return rotate32(x, self.rotary.cos_sin.cpu(), pos, self.rot, "half").to(DT[self.dtype])

    def expect(self, out, q, k, v, plan, starts, p_bits):
        pos = plan.positions
        q, k = self.turn(q, pos), self.turn(k, pos)
        outs, mags, x_abs = [], [], 0.0
        for i, s in enumerate(plan.seqs.tolist()):
            a, b = int(starts[i]), int(starts[i + 1])
            old = self.kv.get(s, (k[:0], v[:0]))
            self.kv[s] = tuple(torch.cat([o, x[a:b]]) for o, x in zip(old, (k, v)))
            n = int(plan.context_lens[i])
            assert self.kv[s][0].shape[0] == n
            seen = np.array([visible(p, n, self.window, self.sinks) for p in range(n - (b - a), n)], bool).reshape(b - a, n)
            o, m, x = attention64(q[a:b].double().numpy(), *(t.double().numpy() for t in self.kv[s]), seen, self.d ** -0.5)
            outs.append(o)
            mags.append(m)
            x_abs = max(x_abs, x)
        check(out, np.concatenate(outs), np.concatenate(mags), x_abs, self.d, int(plan.context_lens.max()), self.dtype, p_bits)

    def prompt(self, seqs, new, prepared=False):
        plan = self.eng.plan_prefill(seqs, new)
        step = self.eng.upload_prefill(plan)
        q, k, v = self.tokens(sum(new))
        dq, dk, dv = (x.to(self.dev) for x in (q, k, v))
        if prepared:
            out = torch.empty_like(dq)
            self.eng.prepare_prefill(dq, dk, dv, step, out)()
        else:
            out = self.eng.prefill(dq, dk, dv, step)
        pkv.check()
        self.expect(out, q, k, v, plan, plan.query_start, 11 if self.dtype == "f16" else 16)

    def fork(self, s):
        c = self.eng.fork(s)
        self.kv[c] = self.kv[s]
        return c

    def step(self, seqs, prepared=False, shared=False, few=True):
        plan = self.eng.plan_step(seqs)
        step = self.eng.upload(plan, shared=shared)
        q, k, v = self.tokens(len(seqs))
        dq, dk, dv = (x.to(self.dev) for x in (q, k, v))
        if prepared:
            out = torch.empty_like(dq)
            p = self.eng.prepare(dq, dk, dv, step, out)
            p()
        else:
            out = self.eng.decode(dq, dk, dv, step)
        pkv.check()
        plain = not shared and self.window > 1 << 39
        self.expect(out, q, k, v, plan, np.arange(len(seqs) + 1),
                    16 if self.dtype == "bf16" and not plain else 22 if few and not plain else 11 if self.dtype == "f16" else 8)
        return step


@pytest.mark.parametrize("dtype,H,Hkv,d,B,window,sinks,rot", [
    ("bf16", 8, 2, 128, 16, 40, 4, 128), ("f16", 6, 3, 64, 8, 17, 0, 32), ("f16", 2, 2, 64, 32, 100, 33, 0), ("bf16", 4, 4, 128, 4, 1, 1, 0)])
def test_a_conversation_in_a_window(cuda_device, dtype, H, Hkv, d, B, window, sinks, rot):
    w = World(cuda_device, dtype, H, Hkv, d, B, window, sinks, rot)
    a, b = w.eng.new_sequence(0), w.eng.new_sequence(0)
    w.prompt([a, b], [137, 20])
    c = w.fork(a)
    for i in range(4):
        w.step([a, b, c], prepared=i % 2 == 1)
    w.prompt([b, c], [145, 1], prepared=True)
    w.step([c, b], prepared=True)


@pytest.mark.parametrize("dtype,H,Hkv,d,B,rot", [("f16", 4, 4, 64, 16, 0), ("bf16", 8, 2, 128, 16, 128)])
def test_samples_of_shared_prompts(cuda_device, dtype, H, Hkv, d, B, rot):
    w = World(cuda_device, dtype, H, Hkv, d, B, rot=rot)
    a, b = w.eng.new_sequence(0), w.eng.new_sequence(0)
    w.prompt([a, b], [150, 70])
    batch = [a] + [w.fork(a) for _ in range(3)] + [b, w.fork(b)]
    for i in range(3):
        step = w.step(batch, prepared=i % 2 == 1, shared=True)
        assert step.groups.prefix.tolist() == [150 // B * B] * 4 + [70 // B * B] * 2
    # every request of a large batch after one prompt
    more = [w.fork(a) for _ in range(30)]
    for i in range(2):
        w.step(batch[:4] + more, prepared=i == 1, shared=True)


def test_a_captured_step_with_groups_and_one_with_a_window_replay(cuda_device):
    for window in (None, 50):
        w = World(cuda_device, "bf16", 8, 2, 128, 16, window, 3 if window else 0)
        a = w.eng.new_sequence(0)
        w.prompt([a], [200])
        batch = [a, w.fork(a), w.fork(a)]
        w.step(batch, shared=window is None)             # the copies on write are done with
        plan = w.eng.plan_step(batch)
        step = w.eng.upload(plan, shared=window is None)
        q, k, v = w.tokens(3)
        staged = StagedInputs({n: (t.shape, t.dtype) for n, t in (("q", q), ("k", k), ("v", v))}, cuda_device)
        out, host = torch.empty_like(q, device=cuda_device), torch.empty_like(q).pin_memory()
        for name, t in (("q", q), ("k", k), ("v", v)):
            staged.host[name].copy_(t)
        graph = GraphStep(staged, lambda s: w.eng.prepare(staged.dev["q"], staged.dev["k"], staged.dev["v"], step, out, stream=s),
                          out, host)
        graph.replay()
        torch.cuda.synchronize()
        first = host.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, host)
        pkv.check()
        w.expect(host, q, k, v, plan, np.arange(4), 16)
