"""Windowed and shared-prefix attention over the paged cache, as they are measured.

Three operators, each in its plain form (elementary torch operations in 32
bits) and through the library's own calls:

    paged_attention_decode_window    one query token per sequence that sees the last `window` tokens
                                     and the first `sinks` ones
    paged_attention_prefill_window   many new tokens per sequence, each with its own such window
    paged_attention_decode_shared    one query token per sequence; sequences of a group share their
                                     first tokens, which are read and multiplied once for the group

Layouts: caches [num_blocks][kv heads][block][head_dim], block tables int32
[seqs][blocks] with -1 past a sequence's end, context lengths int32 [seqs];
query head h reads kv head h / (heads / kv heads).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# -- cases --------------------------------------------------------------------

def listed():
    return [
        # the smallest decode batch: four sequences, where a launch's latency is all there is
        {"name": "window_tiny", "op": "window", "S": 4, "ctx": "1,17,100,300", "window": 64, "sinks": 4, "H": 2,
         "Hkv": 2, "d": 64, "B": 16, "dtype": "f16"},
        # one user's long conversation: one sequence, whose window has to be spread over the GPU
        {"name": "window_one", "op": "window", "S": 1, "ctx": "32768", "window": 4096, "sinks": 4, "H": 32, "Hkv": 8,
         "d": 128, "B": 16, "dtype": "bf16"},
        # the OPT-13B layer batch (lognormal contexts) with a short window: many small pieces of work
        {"name": "window_opt13b", "op": "window", "S": 64, "ctx": "lognormal:500:2048", "window": 255, "sinks": 4,
         "H": 40, "Hkv": 40, "d": 128, "B": 16, "dtype": "f16"},
        # the Llama-2-7B layer batch, a kv head for each query head: the most bytes
        {"name": "window_llama7b", "op": "window", "S": 256, "ctx": "uniform:1:4096", "window": 1024, "sinks": 4,
         "H": 32, "Hkv": 32, "d": 128, "B": 16, "dtype": "f16"},
        # long contexts of grouped heads, of which the window is a small part
        {"name": "window_longgqa", "op": "window", "S": 48, "ctx": "uniform:1000:32768", "window": 4096, "sinks": 16,
         "H": 32, "Hkv": 8, "d": 128, "B": 32, "dtype": "bf16"},
        # the smallest prompt phase: one short prompt
        {"name": "prompt_small", "op": "prompt", "S": 1, "own": "77", "cached": 0, "window": 32, "sinks": 4, "H": 32,
         "Hkv": 8, "d": 128, "B": 16, "dtype": "bf16"},
        # a batch of prompts of uneven lengths, a kv head for each query head
        {"name": "prompt_batch", "op": "prompt", "S": 8, "own": "uniform:512:4096", "cached": 0, "window": 1024,
         "sinks": 4, "H": 32, "Hkv": 32, "d": 128, "B": 16, "dtype": "f16"},
        # two long documents in chunks: what went before lies in the cache
        {"name": "prompt_chunks", "op": "prompt", "S": 2, "own": "4096,4000", "cached": 24577, "window": 4096,
         "sinks": 16, "H": 32, "Hkv": 8, "d": 128, "B": 16, "dtype": "bf16"},
        # the smallest shared decode: one prompt's few samples
        {"name": "shared_small", "op": "shared", "groups": "4", "prefix": "260", "suffix": "uniform:1:40", "H": 8,
         "Hkv": 8, "d": 64, "B": 16, "dtype": "f16"},
        # parallel sampling: 64 prompts of some 500 tokens, four samples of each
        {"name": "shared_sampling", "op": "shared", "groups": "4x64", "prefix": "uniform:497:511",
         "suffix": "uniform:1:256", "H": 32, "Hkv": 32, "d": 128, "B": 16, "dtype": "f16"},
        # one long instruction before every request of a batch, grouped heads
        {"name": "shared_instruction", "op": "shared", "groups": "128", "prefix": "8190", "suffix": "uniform:1:1024",
         "H": 32, "Hkv": 8, "d": 128, "B": 16, "dtype": "bf16"},
        # requests over four long documents, a kv head for each query head
        {"name": "shared_documents", "op": "shared", "groups": "80,33,64,15", "prefix": "uniform:4000:8192",
         "suffix": "uniform:1:512", "H": 32, "Hkv": 32, "d": 128, "B": 32, "dtype": "f16"},
    ]


HEADS = [(2, 2), (8, 1), (8, 8), (12, 4), (14, 2), (16, 2), (32, 4), (32, 8), (32, 32), (40, 40), (48, 4)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w, op = work(c), c["op"]
        b, f = most.get(op, (0, 0))
        most[op] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most[c["op"]][0] and w["flops"] <= most[c["op"]][1] and _tokens(c) * c["Hkv"] * c["d"] <= 1 << 31:
            return c


def _draw(rng):
    op = rng.choice(["window", "prompt", "shared"])
    H, Hkv = rng.choice(HEADS)
    c = {"op": op, "H": H, "Hkv": Hkv, "d": rng.choice([64, 128, 128]), "B": rng.choice([8, 16, 16, 32, 64]),
         "dtype": rng.choice(["f16", "bf16"])}
    if op == "window":
        hi = _log(rng, 1, 32768)
        c |= {"S": _log(rng, 1, 256), "ctx": "uniform:%d:%d" % (rng.randint(0, hi), hi)}
    elif op == "prompt":
        hi = _log(rng, 1, 4096)
        c |= {"S": rng.randint(1, 8), "own": "uniform:%d:%d" % (max(1, hi // 3), hi),
              "cached": rng.choice([0, _log(rng, 1, 16384)])}
    else:
        n = rng.randint(1, 6)
        hi = _log(rng, 1, 8192)
        c |= {"groups": ",".join(str(_log(rng, 1, 128)) for _ in range(n)),
              "prefix": "uniform:%d:%d" % (rng.randint(0, hi), hi), "suffix": "uniform:1:%d" % _log(rng, 1, 1024)}
    if op != "shared":
        c |= {"window": _log(rng, 1, 8192), "sinks": rng.choice([0, 1, 4, 16, rng.randint(0, 300)])}
    return c


def _lengths(spec, n, rng):
    if ":" not in spec:
        return np.array([int(x) for x in spec.split(",")], np.int64)
    kind, a, b = spec.split(":")
    if kind == "uniform":
        return rng.integers(int(a), int(b) + 1, n)
    return np.clip(np.rint(rng.lognormal(math.log(int(a)) - 0.5, 1.0, n)), 1, int(b)).astype(np.int64)


def _shape(case):
    """The lengths of a case, which go with the case: new tokens and contexts of
    each sequence; of a shared case also the groups' starts and prefixes."""
    rng = np.random.default_rng([case["H"], case["Hkv"], case["B"], case["d"]])
    if case["op"] == "window":
        ctx = _lengths(case["ctx"], case["S"], rng)
        return {"new": np.minimum(ctx, 1), "ctx": ctx}
    if case["op"] == "prompt":
        new = _lengths(case["own"], case["S"], rng)
        return {"new": new, "ctx": new + case["cached"]}
    if "x" in case["groups"]:
        each, count = case["groups"].split("x")
        sizes = np.full(int(count), int(each), np.int64)
    else:
        sizes = np.array([int(x) for x in case["groups"].split(",")], np.int64)
    prefix = np.repeat(np.resize(_lengths(case["prefix"], len(sizes), rng), len(sizes)), sizes)
    ctx = prefix + _lengths(case["suffix"], len(prefix), rng)
    # whole blocks are shared; the prefix's last, partly filled one is each sequence's own copy
    return {"new": np.ones_like(ctx), "ctx": ctx, "start": np.concatenate([[0], np.cumsum(sizes)]),
            "prefix": prefix // case["B"] * case["B"]}


def _tokens(case):
    sh = _shape(case)
    return int(sh["ctx"].sum())


def _tables(case, sh, seed):
    """Block tables over a pool whose blocks are handed out in a seeded order."""
    B, ctx = case["B"], sh["ctx"]
    width = max(1, int(-(-ctx.max() // B)))
    t = np.full((len(ctx), width), -1, np.int64)
    live = np.arange(width)[None, :] < (-(-ctx // B))[:, None]
    mine = live.copy()
    if "start" in sh:
        first = np.repeat(sh["start"][:-1], np.diff(sh["start"]))
        shared = np.arange(width)[None, :] < (sh["prefix"] // B)[:, None]
        mine &= ~(shared & (np.arange(len(ctx)) != first)[:, None])
    nb = int(mine.sum()) + 3
    t[mine] = np.random.default_rng(seed).permutation(nb)[:nb - 3]
    if "start" in sh:
        t = np.where(shared, t[first], t)
    return t.astype(np.int32), nb


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    sh = _shape(case)
    tables, nb = _tables(case, sh, seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    st = {"case": case, "tables": dev(tables), "ctx": dev(sh["ctx"]), "mcl": int(sh["ctx"].max()),
          "scale": 1.0 / math.sqrt(d)}
    st["kc"], st["vc"] = (torch.randn(nb, Hkv, B, d, device=DEV, generator=g, dtype=dt) for _ in range(2))
    rows = int(sh["new"].sum()) if case["op"] == "prompt" else len(sh["ctx"])
    st["query"] = torch.randn(rows, H, d, device=DEV, generator=g, dtype=dt)
    st["out"] = torch.empty_like(st["query"])
    if case["op"] == "prompt":
        st |= {"start": dev(np.concatenate([[0], np.cumsum(sh["new"])])), "mql": int(sh["new"].max())}
    if case["op"] == "shared":
        st |= {"group_start": dev(sh["start"]), "prefix": dev(sh["prefix"]), "mpl": int(sh["prefix"].max()),
               "mgs": int(np.diff(sh["start"]).max()), "msl": int((sh["ctx"] - sh["prefix"]).max())}
    return st


# -- the plain forms --------------------------------------------------------------

def _plain_gather(st, token):
    """Keys and values of tokens [S][L] in 32 bits, [S][Hkv][L][d]."""
    B = st["case"]["B"]
    blk = st["tables"].long().gather(1, token // B).clamp(min=0)
    return [pool[blk, :, token % B].float().transpose(1, 2) for pool in (st["kc"], st["vc"])]


def _plain_attend(q, k, v, seen, scale):
    """q [S][Hkv][rows][d]; seen [S][1][rows][L]; a row that sees nothing gives zeros."""
    x = (q @ k.transpose(-1, -2)) * scale
    x = torch.where(seen, x, torch.full((), -math.inf, device=DEV))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    s = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(s == 0, torch.ones_like(s), s)


def _plain_span(st, low, high, length):
    """The tokens that some row of a sequence sees, the first `sinks` and those of
    [low, high), as [S][length] token numbers and which of them there are."""
    t = torch.arange(length, device=DEV)[None, :]
    first = low.clamp(max=st["case"].get("sinks", 0))[:, None]
    token = torch.where(t < first, t, low[:, None] + t - first)
    there = t < first + (high - low)[:, None]
    return torch.where(there, token, torch.zeros_like(token)), there


def _plain_rows(st, seen_of, k, v, token, there):
    """Attention of one query token per sequence."""
    c = st["case"]
    S = st["query"].shape[0]
    q = st["query"].float().view(S, c["Hkv"], c["H"] // c["Hkv"], c["d"])
    v = torch.where(there[:, None, :, None], v, torch.zeros((), device=DEV))
    return _plain_attend(q, k, v, (seen_of(token) & there)[:, None, None, :], st["scale"]).reshape(
        S, c["H"], c["d"]).to(st["query"].dtype)


def _plain_window(st):
    c, ctx = st["case"], st["ctx"].long()
    low = (ctx - c["window"]).clamp(min=0)
    token, there = _plain_span(st, low, ctx, max(1, min(st["mcl"], c["window"] + c["sinks"])))
    k, v = _plain_gather(st, token)
    return _plain_rows(st, lambda t: t < ctx[:, None], k, v, token, there)


def _plain_prompt(st):
    c = st["case"]
    S, Hkv, G, d, n, w = c["S"], c["Hkv"], c["H"] // c["Hkv"], c["d"], st["mql"], c["window"]
    start, ctx = st["start"].long(), st["ctx"].long()
    new = start[1:] - start[:-1]
    low = (ctx - new - w + 1).clamp(min=0)
    token, there = _plain_span(st, low, ctx, min(st["mcl"], n + w + c["sinks"]))
    k, v = _plain_gather(st, token)
    v = torch.where(there[:, None, :, None], v, torch.zeros((), device=DEV))
    j = torch.arange(n, device=DEV)
    row = (start[:-1, None] + j).clamp(max=st["query"].shape[0] - 1)         # [S][n]
    q = st["query"].float()[row].view(S, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * n, d)
    p = ((ctx - new)[:, None] + j)[:, :, None]                                # the rows' positions
    t = token[:, None, :]
    seen = (t <= p) & ((t > p - w) | (t < c["sinks"])) & there[:, None, :] & (j < new[:, None])[:, :, None]
    seen = seen[:, None, None].expand(S, 1, G, n, t.shape[-1]).reshape(S, 1, G * n, -1)
    o = _plain_attend(q, k, v, seen, st["scale"]).view(S, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(S, n, c["H"], d)
    rows = torch.arange(st["query"].shape[0], device=DEV)
    seq = torch.searchsorted(start[1:], rows, right=True)
    return o[seq, rows - start[seq]].to(st["query"].dtype)


def _plain_shared(st):
    ctx = st["ctx"].long()
    token, there = _plain_span(st, torch.zeros_like(ctx), ctx, st["mcl"])
    k, v = _plain_gather(st, token)
    return _plain_rows(st, lambda t: t < ctx[:, None], k, v, token, there)


PLAIN = {"window": _plain_window, "prompt": _plain_prompt, "shared": _plain_shared}


# -- the library's calls ------------------------------------------------------------

def _own_run(st):
    import paged_kv_cache_139_gb300 as pkv
    c = st["case"]
    if c["op"] == "window":
        return pkv.paged_attention_decode_window(st["out"], st["query"], st["kc"], st["vc"], st["tables"], st["ctx"],
                                                 c["window"], c["sinks"], scale=st["scale"], max_context_len=st["mcl"])
    if c["op"] == "prompt":
        return pkv.paged_attention_prefill_window(st["out"], st["query"], st["kc"], st["vc"], st["tables"], st["ctx"],
                                                  st["start"], c["window"], c["sinks"], scale=st["scale"],
                                                  max_query_len=st["mql"])
    return pkv.paged_attention_decode_shared(st["out"], st["query"], st["kc"], st["vc"], st["tables"], st["ctx"],
                                             st["group_start"], st["prefix"], scale=st["scale"],
                                             max_context_len=st["mcl"], max_prefix_len=st["mpl"],
                                             max_group_size=st["mgs"], max_suffix_len=st["msl"])


def run(state):
    if own:
        return _own_run(state)
    return PLAIN[state["case"]["op"]](state)


# -- what a pass cannot do without ----------------------------------------------------

def _visible(ctx, new, window, sinks):
    """Over the new tokens of each sequence: (tokens that some row sees, pairs of a row and a token that it sees)."""
    p0 = ctx - new
    low = np.maximum(0, p0 - window + 1)
    tokens = np.where(new > 0, ctx - low + np.minimum(sinks, low), 0)
    # positions p in [p0, ctx): min(p + 1, window) in the window, and the sinks before it
    def upto(n):                                     # sums over p in [0, n)
        full = np.maximum(0, n - window)
        m = np.minimum(n, window)
        s = np.minimum(full, sinks)                  # p = window + i sees min(i + 1, sinks) sinks
        return m * (m + 1) // 2 + full * window + s * (s + 1) // 2 + (full - s) * sinks
    return tokens, upto(ctx) - upto(p0)


def work(case):
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    sh = _shape(case)
    ctx, new = sh["ctx"], sh["new"]
    if case["op"] == "shared":
        size = np.diff(sh["start"])
        again = int((sh["prefix"][sh["start"][:-1]] * (size - 1)).sum())     # shared tokens, counted once
        tokens, pairs = int(ctx.sum()) - again, int(ctx.sum())
    else:
        t, p = _visible(ctx, new, case["window"], case["sinks"])
        tokens, pairs = int(t.sum()), int(p.sum())
    rows = int(new.sum())
    return {"bytes": tokens * 4 * Hkv * d + 4 * (tokens // B + len(ctx)) + 4 * rows * H * d,
            "flops": 4 * H * d * pairs}


# -- the definitions in 64 bits --------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    G = H // Hkv
    sh = _shape(case)
    # without a window every token up to the row's own is seen
    w, sinks = (case["window"], case["sinks"]) if "window" in case else (1 << 40, 0)
    out = torch.zeros(st["query"].shape, device=DEV, dtype=torch.float64)
    row = 0
    for s, (n, ctx) in enumerate(zip(sh["new"].tolist(), sh["ctx"].tolist())):
        if case["op"] != "prompt":
            row = s
        for a in range(0, n, 512):                    # some rows at a time
            m = min(512, n - a)
            p = torch.arange(ctx - n + a, ctx - n + a + m, device=DEV)
            keep = torch.arange(ctx - n + a + m, device=DEV)
            keep = keep[(keep > ctx - n + a - w) | (keep < sinks)]
            blk = st["tables"][s].long()[keep // B]
            k, v = (x[blk, :, keep % B].double() for x in (st["kc"], st["vc"]))      # [L][Hkv][d]
            x = torch.einsum("jgrd,tgd->grjt", st["query"][row + a:row + a + m].double().view(m, Hkv, G, d), k)
            hidden = (keep[None] > p[:, None]) | ((keep[None] <= p[:, None] - w) & (keep[None] >= sinks))
            x = (x * st["scale"]).masked_fill(hidden, -math.inf)
            out[row + a:row + a + m] = torch.einsum("grjt,tgd->jgrd", torch.softmax(x, -1), v).reshape(m, H, d)
        row += n
    return out
