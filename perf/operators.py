"""The operators of a rotated and of an 8-bit paged KV cache, as they are measured.

Five operators, each in its plain form (elementary torch operations in 32 bits
or more) and through the library's own calls:

    rotary_table                 cos and sin of the rotary angles, scaled for long contexts
    kv_rotary_and_cache          rotate queries and keys, append keys and values to a 16-bit paged cache
    kv_rotary_and_cache_fp8      the same into an e4m3 cache with a scale per block and kv head
    paged_attention_decode_fp8   one query token per sequence over the e4m3 cache
    paged_attention_prefill_fp8  many new tokens per sequence (causal) over the e4m3 cache

Layouts: caches [num_blocks][kv heads][block][head_dim], scales fp32
[num_blocks][kv heads rounded up to even][key, value], block tables int32
[seqs][blocks] with -1 past a sequence's end, slots int64 (block * size + offset).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
MIN_SCALE_EXP = -60          # the smallest block scale is 2^-60


# -- cases --------------------------------------------------------------------

def listed():
    return [
        # the table a model of 2048 positions builds when it loads
        {"name": "table_2k", "op": "table", "n": 2048, "rot": 128, "base": 10000.0, "scaling": "none",
         "factor": 1.0, "orig": 2048},
        # a context of 131,072 positions stretched from 16,384, by parts
        {"name": "table_131k_parts", "op": "table", "n": 131072, "rot": 128, "base": 500000.0,
         "scaling": "by_parts", "factor": 8.0, "orig": 16384},
        # one decode step of the Llama-2-7B layer batch: one token for each of 256 sequences
        {"name": "append_step", "op": "append", "kind": "step", "S": 256, "tokens": 256, "H": 32, "Hkv": 32, "d": 128,
         "rot": 128, "layout": "half", "B": 16, "dtype": "f16", "maxpos": 4096},
        # a batch of prompts, grouped heads, half of the head rotated, pairs interleaved
        {"name": "append_prompt", "op": "append", "kind": "prompt", "S": 21, "tokens": 16381, "H": 32, "Hkv": 8,
         "d": 128, "rot": 64, "layout": "interleaved", "B": 32, "dtype": "bf16", "maxpos": 32768},
        # a decode step of a grouped-head layer into the 8-bit cache, blocks partly filled
        {"name": "append8_step", "op": "append8", "kind": "step", "S": 256, "tokens": 256, "H": 32, "Hkv": 8, "d": 128,
         "rot": 128, "layout": "half", "B": 16, "dtype": "bf16", "maxpos": 4096},
        # a batch of prompts into the 8-bit cache
        {"name": "append8_prompt", "op": "append8", "kind": "prompt", "S": 21, "tokens": 16381, "H": 32, "Hkv": 32,
         "d": 128, "rot": 128, "layout": "half", "B": 16, "dtype": "f16", "maxpos": 4096},
        # the tiny decode batch: what one call costs
        {"name": "decode8_tiny", "op": "decode8", "S": 4, "ctx": "1,17,100,300", "H": 2, "Hkv": 2, "d": 64, "B": 16,
         "dtype": "f16"},
        # the OPT-13B layer batch, ordinary lengths
        {"name": "decode8_opt13b", "op": "decode8", "S": 64, "ctx": "lognormal:500:2048", "H": 40, "Hkv": 40,
         "d": 128, "B": 16, "dtype": "f16"},
        # the Llama-2-7B layer batch: the largest
        {"name": "decode8_llama7b", "op": "decode8", "S": 256, "ctx": "uniform:1:4096", "H": 32, "Hkv": 32, "d": 128,
         "B": 16, "dtype": "f16"},
        # few long contexts with grouped heads: the split over the context
        {"name": "decode8_longgqa", "op": "decode8", "S": 8, "ctx": "uniform:32768:32768", "H": 32, "Hkv": 8,
         "d": 128, "B": 16, "dtype": "bf16"},
        # requests that share a cached 1000-token prefix, each with its own input
        {"name": "prefill8_prefix", "op": "prefill8", "S": 32, "own": "uniform:33:480", "prefix": 1000,
         "shared": True, "H": 32, "Hkv": 32, "d": 128, "B": 16, "dtype": "f16"},
        # one more chunk of two long prompts, grouped heads
        {"name": "prefill8_chunk", "op": "prefill8", "S": 2, "own": "uniform:511:512", "prefix": 15001,
         "shared": False, "H": 32, "Hkv": 8, "d": 128, "B": 32, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "append8", "append8", "decode8", "decode8", "decode8", "prefill8"])
    if op == "table":
        scaling = rng.choice(["none", "linear", "by_parts"])
        n = _log(rng, 100, 131072)
        return {"op": op, "n": n, "rot": rng.choice([16, 32, 64, 96, 128]), "base": rng.choice([1e4, 5e5, 1e6]),
                "scaling": scaling, "factor": 1.0 if scaling == "none" else float(rng.choice([2, 4, 8, 5.5])),
                "orig": max(32, n // rng.choice([2, 4, 8]))}
    d = rng.choice([64, 128, 128])
    B = rng.choice([8, 16, 16, 32, 64])
    dt = rng.choice(["f16", "bf16"])
    H, Hkv = rng.choice([(2, 2), (32, 32), (40, 40), (32, 8), (12, 4), (8, 1), (16, 2), (10, 2), (7, 1), (28, 4)])
    if op in ("append", "append8"):
        kind = rng.choice(["step", "prompt"])
        if kind == "step":
            S = _log(rng, 1, 1024)
            tokens = S
        else:
            tokens = _log(rng, 20, 12000)
            S = rng.randint(1, max(1, min(24, tokens // 16)))
        return {"op": op, "kind": kind, "S": S, "tokens": tokens, "H": H, "Hkv": Hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, 16]), "layout": rng.choice(["half", "interleaved"]), "B": B,
                "dtype": dt, "maxpos": rng.choice([4096, 20000])}
    if op == "decode8":
        S = _log(rng, 1, 256)
        top = min(32768, (1 << 31) // (S * Hkv * d))
        hi = _log(rng, 1, top)
        ctx = "uniform:%d:%d" % (rng.randint(0, hi) if rng.random() < 0.5 else max(1, hi // 2), hi)
        return {"op": op, "S": S, "ctx": ctx, "H": H, "Hkv": Hkv, "d": d, "B": B, "dtype": dt}
    S = rng.randint(1, 16)
    hi = _log(rng, 1, 600)
    return {"op": op, "S": S, "own": "uniform:%d:%d" % (max(1, hi // 3), hi), "prefix": rng.randint(0, 2000),
            "shared": rng.random() < 0.5, "H": H, "Hkv": Hkv, "d": d, "B": B, "dtype": dt}


def _lengths(spec, n, rng):
    if ":" not in spec:
        return np.array([int(x) for x in spec.split(",")], np.int64)
    kind, a, b = spec.split(":")
    if kind == "uniform":
        return rng.integers(int(a), int(b) + 1, n)
    return np.clip(np.rint(rng.lognormal(math.log(int(a)) - 0.5, 1.0, n)), 1, int(b)).astype(np.int64)


def _split(total, n, rng):
    """`total` as n lengths of at least one."""
    cuts = np.sort(rng.choice(np.arange(1, total), n - 1, replace=False)) if n > 1 else np.empty(0, np.int64)
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int64)


def _tables(lens, B, order, width):
    """Block tables over blocks handed out in `order`, sequence by sequence."""
    nb = -(-lens // B)
    t = np.full((len(lens), width), -1, np.int32)
    live = np.arange(width)[None, :] < nb[:, None]
    t[live] = order[:int(nb.sum())]
    return t


def _even(h):
    return h + (h & 1)


def _pool8(nb, hkv, B, d, g):
    x = torch.randn(nb, hkv, B, d, device=DEV, generator=g)
    return x.mul_(100.0).clamp_(-448.0, 448.0).to(F8)


def _pool_scales(nb, hkv, g):
    return 1.0 / (1 << torch.randint(6, 10, (nb, _even(hkv), 2), device=DEV, generator=g)).float()


def _cos_sin(n, rot, base):
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    a = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * torch.pow(base, -2.0 * i / rot)
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _shape(case, seed):
    """The host-side lengths and tables of a case: the lengths go with the case,
    where the blocks lie in the pool with the seed."""
    rng = np.random.default_rng([case["S"], case["H"], case["B"], case["d"]])
    place = np.random.default_rng(seed)
    if case["op"] in ("append", "append8"):
        S, B = case["S"], case["B"]
        if case["kind"] == "step":
            before = rng.integers(0, min(case["maxpos"] - 1, 40 * B) + 1, S)
            new = np.ones(S, np.int64)
        else:
            new = _split(case["tokens"], S, rng)
            before = np.where(rng.random(S) < 0.5, 0, rng.integers(0, 3 * B + 1, S))
        # only the blocks that are written need a place in the pool
        first, last = before // B, (before + new - 1) // B
        nblk = last - first + 1
        nb = int(nblk.sum()) + 3
        order = place.permutation(nb)
        seq = np.repeat(np.arange(S), new)
        j = np.arange(int(new.sum())) - np.repeat(np.cumsum(new) - new, new)
        pos = before[seq] + j
        blk = order[(np.cumsum(nblk) - nblk)[seq] + pos // B - first[seq]]
        return {"nb": nb, "positions": (pos % case["maxpos"]).astype(np.int32),
                "slots": (blk * B + pos % B).astype(np.int64)}
    if case["op"] == "decode8":
        ctx = _lengths(case["ctx"], case["S"], rng)
        width = max(1, int(-(-ctx.max() // case["B"])))
        nb = int((-(-ctx // case["B"])).sum()) + 3
        return {"nb": nb, "ctx": ctx.astype(np.int32), "tables": _tables(ctx, case["B"], place.permutation(nb), width)}
    new = _lengths(case["own"], case["S"], rng)
    ctx = new + case["prefix"]
    B = case["B"]
    width = int(-(-ctx.max() // B))
    nb = int((-(-ctx // B)).sum()) + 3
    tables = _tables(ctx, B, place.permutation(nb), width)
    if case["shared"]:
        tables[:, :case["prefix"] // B] = tables[0, :case["prefix"] // B]
    return {"nb": nb, "ctx": ctx.astype(np.int32), "tables": tables,
            "start": np.concatenate([[0], np.cumsum(new)]).astype(np.int32), "new": new}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "table":
        # a table is made from its parameters: the seed moves the base
        base = case["base"] * (1.0 + (seed % 97) / 1000.0)
        return {"case": case, "base": base,
                "out": torch.empty(case["n"], case["rot"] // 2, 2, device=DEV, dtype=torch.float32)}
    dt = DTYPES[case["dtype"]]
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    sh = _shape(case, seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    st = {"case": case, "nb": sh["nb"]}
    if op in ("append", "append8"):
        T = len(sh["slots"])
        # queries, keys and values as one projection leaves them: slices of its rows
        qkv = torch.randn(T, H + 2 * Hkv, d, device=DEV, generator=g).to(dt)
        st |= {"query": qkv[:, :H], "key": qkv[:, H:H + Hkv], "value": qkv[:, H + Hkv:],
               "positions": dev(sh["positions"]), "slots": dev(sh["slots"]),
               "cos_sin": _cos_sin(case["maxpos"], case["rot"], 10000.0),
               "query_out": torch.empty(T, H, d, device=DEV, dtype=dt)}
        if op == "append":
            st["kc"], st["vc"] = (torch.randn(sh["nb"], Hkv, B, d, device=DEV, generator=g).to(dt) for _ in range(2))
            return st
        st["kc"], st["vc"] = (_pool8(sh["nb"], Hkv, B, d, g) for _ in range(2))
        st["scales"] = _pool_scales(sh["nb"], Hkv, g)
        return st
    st["kc"], st["vc"] = (_pool8(sh["nb"], Hkv, B, d, g) for _ in range(2))
    st["scales"] = _pool_scales(sh["nb"], Hkv, g)
    st |= {"tables": dev(sh["tables"]), "ctx": dev(sh["ctx"]), "mcl": int(sh["ctx"].max()), "scale": 1.0 / math.sqrt(d)}
    rows = case["S"] if op == "decode8" else int(sh["start"][-1])
    st["query"] = torch.randn(rows, H, d, device=DEV, generator=g).to(dt)
    st["out"] = torch.empty_like(st["query"])
    if op == "prefill8":
        st |= {"start": dev(sh["start"]), "mql": int(sh["new"].max())}
    return st


# -- the plain forms --------------------------------------------------------------

def _plain_table(st):
    c = st["case"]
    i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
    theta = torch.pow(st["base"], -2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        theta = theta / c["factor"]
    elif c["scaling"] == "by_parts":
        turns = c["orig"] * theta / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        theta = theta * (keep + (1.0 - keep) / c["factor"])
    a = torch.arange(c["n"], device=DEV, dtype=torch.float64)[:, None] * theta
    return torch.stack([a.cos(), a.sin()], -1).float()


def _plain_rotate(x, cos_sin, positions, rot, layout):
    """x [T][heads][d] in 32 bits, its first `rot` elements rotated by pairs."""
    x = x.float()
    cs = cos_sin[positions.long()]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :rot // 2], r[..., rot // 2:])
    y, z = a * c - b * s, a * s + b * c
    r = torch.stack([y, z], -1).flatten(-2) if layout == "interleaved" else torch.cat([y, z], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_append(st):
    c = st["case"]
    B = c["B"]
    q = _plain_rotate(st["query"], st["cos_sin"], st["positions"], c["rot"], c["layout"]).to(st["query"].dtype)
    k = _plain_rotate(st["key"], st["cos_sin"], st["positions"], c["rot"], c["layout"])
    blk, off = st["slots"] // B, st["slots"] % B
    st["kc"][blk, :, off] = k.to(st["kc"].dtype)
    st["vc"][blk, :, off] = st["value"]
    return {"query": q, "key_cache": st["kc"], "value_cache": st["vc"]}


def _pow2_scale(amax):
    """The smallest 2^e with amax <= 448 * 2^e (e >= MIN_SCALE_EXP)."""
    m, e = torch.frexp(amax)                       # amax = m * 2^e, m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)      # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_SCALE_EXP)).clamp(min=MIN_SCALE_EXP)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)      # 2^e by its bits


def _plain_append8(st):
    c = st["case"]
    B, Hkv = c["B"], c["Hkv"]
    q = _plain_rotate(st["query"], st["cos_sin"], st["positions"], c["rot"], c["layout"]).to(st["query"].dtype)
    k = _plain_rotate(st["key"], st["cos_sin"], st["positions"], c["rot"], c["layout"])
    v = st["value"].float()
    blk, off = st["slots"] // B, st["slots"] % B
    # the scale that each block needs for the new tokens, and what it has (none where offset 0 starts it anew)
    need = torch.stack([k.abs().amax(-1), v.abs().amax(-1)], -1)
    top = torch.full((st["nb"], Hkv, 2), -1.0, device=DEV)
    top.scatter_reduce_(0, blk[:, None, None].expand_as(need), need, "amax")
    fresh = torch.zeros(st["nb"], device=DEV).index_put_((blk,), (off == 0).float(), accumulate=True) > 0
    scales = st["scales"][:, :Hkv]
    old = torch.where(fresh[:, None, None], torch.zeros_like(scales), scales)
    new = torch.where(top >= 0, torch.maximum(old, _pow2_scale(top.clamp(min=0.0))), scales)
    ratio = torch.where(fresh[:, None, None], torch.ones_like(new), scales / new)
    tok = new[blk]
    for x, pool, i in ((k, st["kc"], 0), (v, st["vc"], 1)):
        pool.copy_((pool.float() * ratio[:, :, i, None, None]).to(F8))      # the other rows, at the block's new scale
        pool.view(torch.uint8)[blk, :, off] = (x / tok[:, :, i, None]).to(F8).view(torch.uint8)
    st["scales"][:, :Hkv] = new
    return {"query": q, "key_cache": st["kc"], "value_cache": st["vc"], "scales": st["scales"]}


def _plain_gather(st):
    """Each sequence's keys and values in 32 bits, [S][Hkv][tokens][d]."""
    c = st["case"]
    t = st["tables"].clamp(min=0).long()
    got = []
    for pool, i in ((st["kc"], 0), (st["vc"], 1)):
        x = pool.view(torch.uint8)[t].view(F8).float()                       # [S][MB][Hkv][B][d]
        x = x * st["scales"][t][:, :, :c["Hkv"], i, None, None]
        got.append(x.transpose(1, 2).flatten(2, 3))
    return got


def _plain_attend(q, k, v, seen, scale):
    """q [S][Hkv][rows][d]; seen [S][1][rows][tokens]; a row that sees nothing gives zeros."""
    x = (q @ k.transpose(-1, -2)) * scale
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    s = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(s == 0, torch.ones_like(s), s)


def _plain_decode8(st):
    c = st["case"]
    k, v = _plain_gather(st)
    q = st["query"].float().view(c["S"], c["Hkv"], c["H"] // c["Hkv"], c["d"])
    seen = torch.arange(k.shape[2], device=DEV)[None, :] < st["ctx"][:, None]
    v = torch.where(seen[:, None, :, None], v, torch.zeros_like(v))
    return _plain_attend(q, k, v, seen[:, None, None, :], st["scale"]).reshape(c["S"], c["H"], c["d"]).to(
        st["query"].dtype)


def _plain_prefill8(st):
    c = st["case"]
    S, Hkv, G, d, n = c["S"], c["Hkv"], c["H"] // c["Hkv"], c["d"], st["mql"]
    k, v = _plain_gather(st)
    start, ctx = st["start"].long(), st["ctx"].long()
    new = start[1:] - start[:-1]
    j = torch.arange(n, device=DEV)
    row = (start[:-1, None] + j).clamp(max=st["query"].shape[0] - 1)         # [S][n]
    live = j[None, :] < new[:, None]
    q = st["query"].float()[row].view(S, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * n, d)
    t = torch.arange(k.shape[2], device=DEV)
    seen = (t <= (ctx - new)[:, None, None] + j[None, :, None]) & live[:, :, None]   # [S][n][tokens]
    v = torch.where((t < ctx[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = _plain_attend(q, k, v, seen[:, None].expand(S, G, n, t.numel()).reshape(S, 1, G * n, -1), st["scale"])
    o = o.view(S, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(S, n, c["H"], d)
    seq = torch.searchsorted(start[1:], torch.arange(st["query"].shape[0], device=DEV), right=True)
    return o[seq, torch.arange(st["query"].shape[0], device=DEV) - start[seq]].to(st["query"].dtype)


PLAIN = {"table": _plain_table, "append": _plain_append, "append8": _plain_append8, "decode8": _plain_decode8,
         "prefill8": _plain_prefill8}


# -- the library's calls ------------------------------------------------------------

def _own_run(st):
    import paged_kv_cache_139_gb300 as pkv
    c = st["case"]
    if c["op"] == "table":
        return pkv.rotary_table(c["n"], c["rot"], base=st["base"], scaling=c["scaling"], factor=c["factor"],
                                original_positions=c["orig"], out=st["out"])
    if c["op"] == "append":
        q = pkv.kv_rotary_and_cache(st["query"], st["key"], st["value"], st["cos_sin"], st["positions"], st["kc"],
                                    st["vc"], st["slots"], layout=c["layout"], query_out=st["query_out"])
        return {"query": q, "key_cache": st["kc"], "value_cache": st["vc"]}
    if c["op"] == "append8":
        q = pkv.kv_rotary_and_cache_fp8(st["query"], st["key"], st["value"], st["cos_sin"], st["positions"], st["kc"],
                                        st["vc"], st["scales"], st["slots"], layout=c["layout"],
                                        query_out=st["query_out"])
        return {"query": q, "key_cache": st["kc"], "value_cache": st["vc"], "scales": st["scales"]}
    if c["op"] == "decode8":
        return pkv.paged_attention_decode_fp8(st["out"], st["query"], st["kc"], st["vc"], st["scales"], st["tables"],
                                              st["ctx"], scale=st["scale"], max_context_len=st["mcl"])
    return pkv.paged_attention_prefill_fp8(st["out"], st["query"], st["kc"], st["vc"], st["scales"], st["tables"],
                                           st["ctx"], st["start"], scale=st["scale"], max_query_len=st["mql"],
                                           max_context_len=st["mcl"])


def run(state):
    if own:
        return _own_run(state)
    return PLAIN[state["case"]["op"]](state)


# -- what a pass cannot do without ----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": case["n"] * case["rot"] * 4, "flops": 0}
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    if op in ("append", "append8"):
        T, cache = case["tokens"], 2 if op == "append" else 1
        row = (2 * H + 2 * Hkv) * d * 2 + 2 * Hkv * d * cache + case["rot"] * 4 + 12
        scales = 0 if op == "append" else 16 * Hkv * (T if case["kind"] == "step" else -(-T // B))
        return {"bytes": T * row + scales, "flops": T * (H + Hkv) * case["rot"] * 3}
    sh = _shape(case, 0)
    ctx = sh["ctx"].astype(np.int64)
    nblk = int((-(-ctx // B)).sum())
    if op == "decode8":
        kv = int(ctx.sum()) * 2 * Hkv * d
        return {"bytes": kv + nblk * (4 + 8 * Hkv) + 4 * case["S"] * H * d, "flops": 4 * H * d * int(ctx.sum())}
    new = sh["new"]
    tokens = int(ctx.sum()) - ((case["S"] - 1) * (case["prefix"] // B) * B if case["shared"] else 0)
    pairs = int((new * (ctx - new) + new * (new + 1) // 2).sum())
    return {"bytes": tokens * 2 * Hkv * d + nblk * 4 + tokens // B * 8 * Hkv + 4 * int(new.sum()) * H * d,
            "flops": 4 * H * d * pairs}


# -- the definitions in 64 bits --------------------------------------------------------

def _rotate64(x, st, c):
    """Each pair (a, b) as a complex number times cos + i sin, element by element."""
    x = x.double().clone()
    cs = torch.view_as_complex(st["cos_sin"].double())[st["positions"].long()]
    h = c["rot"] // 2
    i = torch.arange(h, device=DEV)
    ia, ib = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + h)
    z = torch.complex(x[:, :, ia], x[:, :, ib]) * cs[:, None, :]
    x[:, :, ia], x[:, :, ib] = z.real, z.imag
    return x


def _two_to(e):
    """2^e in 64 bits for whole e, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """To the e4m3 grid: three bits after the leading one, exponents from -6, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = _two_to(e - 3.0)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    op, c = case["op"], case
    if op == "table":
        out = torch.empty(c["n"], c["rot"] // 2, 2, device=DEV, dtype=torch.float64)
        p = torch.arange(c["n"], device=DEV, dtype=torch.float64)
        for i in range(c["rot"] // 2):
            w = st["base"] ** (-2.0 * i / c["rot"])
            if c["scaling"] != "none":
                r = w * c["orig"] / (2 * math.pi)
                y = 0.0 if c["scaling"] == "linear" else min(1.0, max(0.0, (r - 1.0) / 31.0))
                w = (1.0 - y) * w / c["factor"] + y * w
            out[:, i, 0], out[:, i, 1] = torch.cos(p * w), torch.sin(p * w)
        return out
    H, Hkv, d, B = c["H"], c["Hkv"], c["d"], c["B"]
    if op in ("append", "append8"):
        q, k, v = _rotate64(st["query"], st, c), _rotate64(st["key"], st, c), st["value"].double()
        slots = st["slots"].cpu().numpy()
        kc, vc = st["kc"].double(), st["vc"].double()
        blk, off = torch.from_numpy(slots // B).to(DEV), torch.from_numpy(slots % B).to(DEV)
        if op == "append":
            kc[blk, :, off], vc[blk, :, off] = k, v
            return {"query": q, "key_cache": kc, "value_cache": vc}
        sc = st["scales"].double()
        order = np.argsort(slots // B, kind="stable")
        ids, first = np.unique((slots // B)[order], return_index=True)
        lens = torch.from_numpy(np.diff(np.append(first, len(order)))).to(DEV)
        ids_t, order_t = torch.from_numpy(ids).to(DEV), torch.from_numpy(order).to(DEV)
        anew = torch.from_numpy(np.isin(ids, (slots // B)[slots % B == 0])).to(DEV)
        for x, pool, i in ((k, kc, 0), (v, vc, 1)):
            am = torch.segment_reduce(x.abs().amax(-1)[order_t], "max", lengths=lens)       # [blocks][Hkv]
            e = torch.ceil(torch.log2(am / 448.0)).clamp(min=MIN_SCALE_EXP)
            e = torch.where(am <= 448.0 * _two_to(e - 1), e - 1, e).clamp(min=MIN_SCALE_EXP)
            had = sc[ids_t, :Hkv, i]
            now = torch.where(anew[:, None], _two_to(e), torch.maximum(had, _two_to(e)))
            pool[ids_t] = torch.where(anew[:, None, None, None], pool[ids_t],
                                      _e4m3(pool[ids_t] * (had / now)[:, :, None, None]))
            sc[ids_t, :Hkv, i] = now
            pool[blk, :, off] = _e4m3(x / sc[blk, :Hkv, i][:, :, None])
        return {"query": q, "key_cache": kc, "value_cache": vc, "scales": sc}
    G = H // Hkv
    tables, ctx = st["tables"].long(), st["ctx"].tolist()
    start = list(range(c["S"] + 1)) if op == "decode8" else st["start"].tolist()
    out = torch.zeros(st["query"].shape, device=DEV, dtype=torch.float64)
    for s in range(c["S"]):
        n, a, b = ctx[s], start[s], start[s + 1]
        if n == 0:
            continue
        t = tables[s, :-(-n // B)]
        kv = [(p[t].double() * st["scales"][t][:, :Hkv, i].double()[:, :, None, None]).transpose(0, 1).reshape(
            Hkv, -1, d)[:, :n] for p, i in ((st["kc"], 0), (st["vc"], 1))]
        x = torch.einsum("jgrd,gtd->grjt", st["query"][a:b].double().view(b - a, Hkv, G, d), kv[0]) * st["scale"]
        late = torch.arange(n, device=DEV)[None, :] > (n - (b - a) + torch.arange(b - a, device=DEV))[:, None]
        x.masked_fill_(late, -math.inf)
        out[a:b] = torch.einsum("grjt,gtd->jgrd", torch.softmax(x, -1), kv[1]).reshape(b - a, H, d)
    return out
