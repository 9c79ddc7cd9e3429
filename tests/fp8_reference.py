"""The 8-bit cache and the rotary rotation from their definitions, on the CPU.

Codes are compared exactly: the rotation is the formula in 32 bits, each
product and sum rounded on its own (which is what the library documents), a
block's scale is a power of two, so code = round(x / scale) has one answer.
Attention is in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn


def e4m3_values() -> np.ndarray:
    """The 256 codes' values from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c >> 7, -v, v)


def to_code(x) -> np.ndarray:
    """Nearest code of each fp32 value, ties to the even code, magnitudes above 448 to 448, NaN to NaN."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()[:127]                        # 0 .. 448 in code order
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, np.nan_to_num(a)), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == 0, 0, code) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def pow2_scale(amax: float) -> float:
    if not amax > 0:
        return 2.0 ** -60
    e = math.ceil(math.log2(amax / 448.0)) - 2
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -60)


def rotate32(x: torch.Tensor, cos_sin: torch.Tensor, positions, rot: int, layout: str) -> torch.Tensor:
    """x [T][h][d] on the CPU; fp32 result of the formula, every operation rounded on its own."""
    x = x.float().clone()
    if not rot:
        return x
    cs = cos_sin[torch.as_tensor(np.asarray(positions), dtype=torch.long)][:, None]
    c, s = cs[..., 0], cs[..., 1]
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia] = a * c - b * s
    x[..., ib] = a * s + b * c
    return x


class RefCache8:
    """Codes uint8 [NB][Hkv][B][d] for keys and values, scales fp32 [NB][Hs][2]."""

    def __init__(self, k, v, scales):
        self.codes = [x.cpu().view(torch.uint8).numpy().copy() for x in (k, v)]
        self.scales = scales.cpu().numpy().copy()
        self.B = self.codes[0].shape[2]

    def append(self, k32, v32, slots):
        """k32, v32 fp32 [T][Hkv][d], rotated; one call."""
        values = e4m3_values()
        by_block: dict = {}
        for t, s in enumerate(slots):
            if s >= 0:
                by_block.setdefault(int(s) // self.B, []).append(t)
        for b, toks in by_block.items():
            offs = [int(slots[t]) % self.B for t in toks]
            for i, x32 in enumerate((k32, v32)):
                x = np.asarray(x32)[toks].astype(np.float32)                  # [n][Hkv][d]
                for h in range(x.shape[1]):
                    mag = np.abs(x[:, h])
                    mag = np.minimum(mag[~np.isnan(mag)], np.float32(3.4028235e38))
                    need = np.float32(pow2_scale(float(mag.max()) if mag.size else 0.0))
                    had = np.float32(0.0) if 0 in offs else self.scales[b, h, i]
                    new = max(had, need)
                    if 0 not in offs and new != had:
                        rest = [o for o in range(self.B) if o not in offs]
                        ratio = np.float32(had / new)
                        old = values[self.codes[i][b, h, rest]]
                        self.codes[i][b, h, rest] = to_code(old.astype(np.float32) * ratio)
                    self.scales[b, h, i] = new
                    with np.errstate(invalid="ignore"):
                        self.codes[i][b, h, offs] = to_code(x[:, h] / new)

    def values(self, i):
        """[NB][Hkv][B][d] in 64 bits."""
        hkv = self.codes[i].shape[1]
        return e4m3_values()[self.codes[i]] * self.scales[:, :hkv, i, None, None].astype(np.float64)


def attention64(q, kvals, vvals, table, n, scale):
    """q [rows][H][d] fp64: the last `rows` of n tokens, causal.  kvals, vvals
    [NB][Hkv][B][d].  Returns (out, dx, vmax): the result, a bound of each
    score's error per unit of accumulation error, and the largest value."""
    rows, H, d = q.shape
    Hkv, B = kvals.shape[1], kvals.shape[2]
    blocks = table[:-(-n // B)]
    k = kvals[blocks].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n]
    v = vvals[blocks].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n]
    G = H // Hkv
    qg = q.reshape(rows, Hkv, G, d)
    x = np.einsum("rgjd,gtd->rgjt", qg, k) * scale
    mag = float(np.max(np.einsum("rgjd,gtd->rgjt", np.abs(qg), np.abs(k)))) * abs(scale)
    pos = n - rows + np.arange(rows)
    x = np.where(np.arange(n)[None, :] <= pos[:, None], x.transpose(1, 2, 0, 3), -np.inf)
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    out = np.einsum("gjrt,gtd->rgjd", p, v).reshape(rows, H, d)
    return out, mag, float(np.abs(v).max())


def attention_tolerance(out, mag, vmax, n, d, eps, p_bits):
    """|got - want|: half a step of the output type; each score off by the
    fp32 accumulation of d products in steps of 16 (an MMA adds with up to 2^-22
    relative to the magnitudes summed) and its scaling and exponent, twice
    (weight and sum); the probabilities' rounding; the sum over n tokens in
    steps of 16."""
    u = 2.0 ** -22
    dx = (d / 16 + 8) * u * mag
    return eps / 2 * np.abs(out) + vmax * (2 * dx + 2.0 ** -p_bits + (n / 16 + 32) * u)
