"""Windowed and shared-prefix calls over tens of thousands of sequences on the
GPU, most of them of a token or two: what has no work costs a call no time."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from span_reference import DT, attention64, check, visible

pytestmark = pytest.mark.gpu


def windowed(q, k, v, window, sinks):
    """64-bit outputs of a whole prompt, some rows at a time over the tokens that they see."""
    n, outs, mags, x_abs = len(q), [], [], 0.0
    for a in range(0, n, 512):
        rows = range(a, min(n, a + 512))
        keep = [t for t in range(rows[-1] + 1) if t < sinks or t > a - window]
        seen = np.array([visible(p, rows[-1] + 1, window, sinks)[keep] for p in rows])
        o, m, x = attention64(q[a:rows[-1] + 1], k[keep], v[keep], seen, q.shape[-1] ** -0.5)
        outs.append(o)
        mags.append(m)
        x_abs = max(x_abs, x)
    return np.concatenate(outs), np.concatenate(mags), x_abs


@pytest.mark.parametrize("H,Hkv,dtype", [(2, 1, "bf16"), (2, 2, "f16")])
@pytest.mark.parametrize("bounded", [False, True])
def test_long_prompts_beside_tokens_of_thousands(cuda_device, H, Hkv, dtype, bounded):
    """60,002 sequences: one new token each, but for prompts of 3,000 and of 10,001 tokens.  Without a bound on the
    lengths the batch could hold one prompt of all tokens."""
    S, d, B, window, sinks = 60002, 64, 64, 300, 4
    new = np.ones(S, np.int64)
    long = {7: 3000, 40001: 10001}
    for s, n in long.items():
        new[s] = n
    g = torch.Generator().manual_seed(H + Hkv)
    NB = 64 + sum(-(-n // B) for n in long.values())
    kc, vc = (torch.randn(NB, Hkv, B, d, generator=g).to(DT[dtype]) for _ in range(2))
    tables = np.full((S, -(-max(long.values()) // B)), -1, np.int32)
    tables[:, 0] = np.arange(S) % 64
    at = 64
    for s, n in long.items():
        tables[s, :-(-n // B)] = range(at, at + -(-n // B))
        at += -(-n // B)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn(int(start[-1]), H, d, generator=g).to(DT[dtype])
    dev = lambda a: torch.as_tensor(a).to(cuda_device)  # noqa: E731
    out = torch.full_like(q, math.nan).to(cuda_device)
    pkv.paged_attention_prefill_window(out, dev(q), dev(kc), dev(vc), dev(tables), dev(new.astype(np.int32)), dev(start),
                                       window, sinks, max_query_len=max(long.values()) if bounded else 0)
    pkv.check()
    out = out.cpu()
    single = np.flatnonzero(new == 1)
    # a row that sees one token gives its value: both weights are the same number
    want = vc[torch.from_numpy(tables[single, 0]).long(), :, 0].repeat_interleave(H // Hkv, 1)
    assert torch.equal(out[torch.from_numpy(start[single]).long()], want)
    for s, n in long.items():
        flat = lambda x: x[tables[s, :-(-n // B)]].transpose(1, 2).reshape(-1, Hkv, d)[:n].double().numpy()  # noqa: E731
        rows = slice(int(start[s]), int(start[s]) + n)
        check(out[rows], *windowed(q[rows].double().numpy(), flat(kc), flat(vc), window, sinks), d, n, dtype,
              16 if dtype == "bf16" else 11)


@pytest.mark.parametrize("bounded", [False, True])
def test_shared_prompts_beside_thousands_of_strangers(cuda_device, bounded):
    """60,000 sequences of a token each around groups of 100 and 300 after 1,000 and 601 shared tokens.  Without
    bounds every group could hold all sequences."""
    H, Hkv, d, B, dtype = 8, 2, 64, 64, "bf16"
    sizes = [1] * 20000 + [100] + [1] * 30000 + [300] + [1] * 10000
    first = {20000: (100, 1000), 50100: (300, 601)}          # a group's first sequence: its size and prefix
    S = sum(sizes)
    rng = np.random.default_rng(5)
    ctx, prefix, width = np.ones(S, np.int32), np.zeros(S, np.int32), 17
    tables = np.full((S, width), -1, np.int32)
    tables[:, 0] = np.arange(S) % 64
    at = 64
    for s, (n, p) in first.items():
        own = rng.integers(1, 40, n)
        ctx[s:s + n], prefix[s:s + n] = p + own, p
        for i in range(n):                                   # a prefix's last, partly filled block is read through
            shared = -(-p // B) if i == 0 else p // B        # the first sequence's table; the others' own hold anything
            if i:
                tables[s + i, :shared] = tables[s, :shared]
            need = -(-int(ctx[s + i]) // B)
            start = 0 if i == 0 else shared
            tables[s + i, start:need] = range(at, at + need - start)
            at += need - start
    g = torch.Generator().manual_seed(9)
    kc, vc = (torch.randn(at, Hkv, B, d, generator=g).to(DT[dtype]) for _ in range(2))
    q = torch.randn(S, H, d, generator=g).to(DT[dtype])
    dev = lambda a: torch.as_tensor(np.ascontiguousarray(a) if isinstance(a, np.ndarray) else a).to(cuda_device)  # noqa: E731
    out = torch.full_like(q, math.nan).to(cuda_device)
    gs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    kw = dict(max_prefix_len=1000, max_group_size=300, max_suffix_len=39) if bounded else {}
    pkv.paged_attention_decode_shared(out, dev(q), dev(kc), dev(vc), dev(tables), dev(ctx), dev(gs), dev(prefix), **kw)
    pkv.check()
    out = out.cpu()
    lone = torch.from_numpy(np.flatnonzero(ctx == 1))
    assert torch.equal(out[lone], vc[torch.from_numpy(tables[lone.numpy(), 0]).long(), :, 0].repeat_interleave(H // Hkv, 1))
    for s, (n, p) in first.items():
        outs, mags, x_abs = [], [], 0.0
        for i in range(s, s + n):
            c = int(ctx[i])
            read = tables[i].copy()
            read[:p // B] = tables[s, :p // B]
            flat = lambda x, t: x[t[:-(-c // B)]].transpose(1, 2).reshape(-1, Hkv, d)[:c].double().numpy()  # noqa: E731
            k, v = flat(kc, read), flat(vc, read)
            tail = slice(p // B * B, p)                      # the first sequence's rows of the block that is not full
            for own, pool in ((k, kc), (v, vc)):
                own[tail] = pool[tables[s, p // B], :, :p % B].transpose(0, 1).double().numpy()
            o, m, x = attention64(q[i:i + 1].double().numpy(), k, v, np.ones((1, c), bool), d ** -0.5)
            outs.append(o)
            mags.append(m)
            x_abs = max(x_abs, x)
        check(out[s:s + n], np.concatenate(outs), np.concatenate(mags), x_abs, d, int(ctx.max()), dtype, 16)
