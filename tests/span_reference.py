"""Windowed and shared-prefix attention from its definition, in 64 bits on the
CPU, with bounds on what the kernels' roundings may leave.

A pool's blocks outside a case hold NaN, and so do the tokens that no row of
their sequence sees where the definition says they have no effect."""
from __future__ import annotations

import math

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def visible(p: int, n: int, window: int, sinks: int) -> np.ndarray:
    """Which of n tokens the row at position p sees."""
    t = np.arange(n)
    return (t <= p) & ((t > p - window) | (t < sinks))


def attention64(q, k, v, seen, scale):
    """q [r][H][d], k and v [n][Hkv][d], seen [r][n]: (out, sum of p |v|, the largest sum of |scale q_i k_i|)."""
    r, H, d = q.shape
    g = H // k.shape[1]
    out, mag, x_abs = np.zeros((r, H, d)), np.zeros((r, H, d)), 0.0
    for h in range(H):
        kh, vh = k[:, h // g], v[:, h // g]
        x = q[:, h] @ kh.T * scale
        x_abs = max(x_abs, float((np.abs(q[:, h]) @ np.abs(kh).T * abs(scale))[seen].max(initial=0.0)))
        x = np.where(seen, x, -np.inf)
        m = x.max(1, initial=-np.inf, keepdims=True)
        p = np.exp(x - np.where(np.isinf(m), 0.0, m))
        l = p.sum(1, keepdims=True)
        p = p / np.where(l == 0, 1.0, l)
        out[:, h], mag[:, h] = p @ vh, p @ np.abs(vh)
    return out, mag, x_abs


def tolerance(out, mag, x_abs, d, n, dtype, p_bits, v_max):
    """The output's rounding (half a step of its type); the probabilities' (2^-p_bits of
    each; of those in 11 bits also what falls below fp16's least number, 2^-25); a score's
    d products and sums in 32 bits (2^-24 of the sum of their magnitudes each) as a relative
    error of its exponential, in numerator and denominator; exponentials, sums and the
    division (16 times 2^-22)."""
    half = torch.finfo(DT[dtype]).eps / 2
    least = torch.finfo(DT[dtype]).smallest_normal * half if dtype == "f16" else 0.0
    rel = 2.0 ** -p_bits + 2 * d * 2.0 ** -24 * x_abs + 16 * 2.0 ** -22
    return half * np.abs(out) + mag * rel + least + (n * 2.0 ** -25 * v_max if p_bits == 11 else 0.0)


def check(got, out, mag, x_abs, d, n, dtype, p_bits, v_max=6.0):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{int((~np.isfinite(got)).sum())} of {got.size} not finite"
    tol = tolerance(out, mag, x_abs, d, n, dtype, p_bits, v_max)
    off = np.abs(got - out)
    worst = float((off / tol).max(initial=0.0))
    assert worst <= 1.0, f"worst {worst:.3f} of its tolerance at {np.unravel_index((off / tol).argmax(), off.shape)}"
    if got.size >= 4096:
        # over many elements roundings add up as their squares do: each at most a third of half a step
        # squared, the probabilities' in 11 bits as much again as the output's
        rms = np.linalg.norm(got - out) / np.linalg.norm(out)
        half = torch.finfo(DT[dtype]).eps / 2
        assert rms <= half * (1.0 if p_bits > 11 else 1.4) / math.sqrt(3) * 1.2, f"rms error {rms / half:.3f} half steps"


class SpanCase:
    """Sequences of given context lengths, `new` of each as query rows (the last
    tokens of its context), over a shuffled pool.  groups: sizes of consecutive
    groups, prefix: their shared tokens (the full blocks are the same ones, a rest
    is copied)."""

    def __init__(self, dev, ctx, H, Hkv, d, B, dtype="f16", new=None, groups=None, prefix=None, seed=0, extra=5,
                 offset=0):
        rng = np.random.default_rng(seed)
        self.dev, self.H, self.Hkv, self.d, self.B, self.dtype = dev, H, Hkv, d, B, dtype
        self.ctx = np.asarray(ctx, np.int32)
        self.new = np.asarray(new if new is not None else np.minimum(self.ctx, 1), np.int64)
        S = len(ctx)
        nblk = -(-self.ctx // B)
        width = max(1, int(nblk.max()))
        self.groups = list(groups) if groups else None
        first, pre = np.arange(S), np.zeros(S, np.int64)
        if groups:
            start = np.concatenate([[0], np.cumsum(groups)])
            assert start[-1] == S
            first = np.repeat(start[:-1], groups)
            pre = np.repeat(np.asarray(prefix), groups)
            self.start, self.prefix = start.astype(np.int32), pre.astype(np.int32)
        self.kv = []                                     # per sequence: k, v [n][Hkv][d] (64 bits, of 16-bit numbers)
        draw = lambda n: torch.from_numpy(rng.standard_normal((n, Hkv, d)).astype(np.float32)).to(DT[dtype])  # noqa: E731
        for s in range(S):
            n, f, p = int(self.ctx[s]), int(first[s]), int(pre[s])
            k, v = draw(n), draw(n)
            if f != s and p:
                k[:p], v[:p] = self.kv[f][0][:p], self.kv[f][1][:p]
            self.kv.append((k, v))
        own = nblk.copy()
        for s in range(S):
            if first[s] != s:
                own[s] -= pre[s] // B
        NB = int(own.sum()) + extra
        order = rng.permutation(NB) + offset
        self.tables = np.full((S, width), -1, np.int32)
        at = 0
        for s in range(S):
            share = int(pre[s]) // B if first[s] != s else 0
            self.tables[s, :share] = self.tables[first[s], :share]
            self.tables[s, share:nblk[s]] = order[at:at + own[s]]
            at += own[s]
        self.NB = NB + offset
        nan = lambda: torch.full((NB, Hkv, B, d), math.nan, dtype=DT[dtype])  # noqa: E731
        pools = [nan(), nan()]
        for s in range(S):
            for i in range(2):
                for j in range(int(nblk[s])):
                    rows = self.kv[s][i][j * B:(j + 1) * B]
                    pools[i][self.tables[s, j] - offset, :, :rows.shape[0]] = rows.transpose(0, 1)
        self.pools = pools
        self.q = torch.from_numpy(rng.standard_normal((int(self.new.sum()), H, d)).astype(np.float32)).to(DT[dtype])
        self.offset = offset

    def spoil(self, window, sinks):
        """NaN in every token that no row of its sequence sees; entries of blocks with no other token out of range."""
        for s in range(len(self.ctx)):
            n = int(self.ctx[s])
            seen = np.zeros(n, bool)
            for p in range(n - int(self.new[s]), n):
                seen |= visible(p, n, window, sinks)
            for t in np.flatnonzero(~seen):
                for x in self.pools:
                    x[self.tables[s, t // self.B] - self.offset, :, t % self.B] = math.nan
            for j in range(-(-n // self.B)):
                if not seen[j * self.B:(j + 1) * self.B].any():
                    self.tables[s, j] = (-1, 1 << 30, -(1 << 31))[j % 3]
        return self

    def upload(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(self.dev)  # noqa: E731
        if self.offset:
            shape = (self.NB, *self.pools[0].shape[1:])
            self.kc, self.vc = (torch.empty(shape, dtype=DT[self.dtype], device=self.dev) for _ in range(2))
            for big, x in zip((self.kc, self.vc), self.pools):
                big[self.offset:] = x.to(self.dev)
        else:
            self.kc, self.vc = (x.to(self.dev) for x in self.pools)
        self.t, self.c, self.qd = t(self.tables), t(self.ctx), self.q.to(self.dev)
        self.qs = t(np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32))
        if self.groups:
            self.gs, self.pl = t(self.start), t(self.prefix)
        self.out = torch.full_like(self.qd, math.nan)
        return self

    def expect(self, window=1 << 40, sinks=0, scale=None):
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        outs, mags, x_abs, row = [], [], 0.0, 0
        for s in range(len(self.ctx)):
            n, r = int(self.ctx[s]), int(self.new[s])
            seen = np.array([visible(p, n, window, sinks) for p in range(n - r, n)], bool).reshape(r, n)
            k, v = (x.double().numpy() for x in self.kv[s])
            o, m, x = attention64(self.q[row:row + r].double().numpy(), k, v, seen, scale)
            row += r
            outs.append(o)
            mags.append(m)
            x_abs = max(x_abs, x)
        return np.concatenate(outs), np.concatenate(mags), x_abs
