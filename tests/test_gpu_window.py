"""Attention with a sliding window and sinks on the GPU against 64 bits: single
tokens and prompts, at the lengths, windows and blocks where a tile or a stage
begins, ends or holds nothing that a row sees."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from span_reference import SpanCase, check

pytestmark = pytest.mark.gpu
ALL = 1 << 30
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 300]


def bits(dtype):
    return 22 if dtype == "f16" else 16


def decode(c, window, sinks, out=None, **kw):
    out = torch.full_like(c.qd, math.nan) if out is None else out
    return pkv.paged_attention_decode_window(out, c.qd, c.kc, c.vc, c.t, c.c, window, sinks, **kw)


def rows_of(c):
    """One query row for every sequence, also those without tokens."""
    q = torch.randn(len(c.ctx), c.H, c.d, generator=torch.Generator().manual_seed(3)).to(c.q.dtype)
    c.q = q
    return c


def decode_case(dev, ctx, *args, window, sinks, spoil=True, **kw):
    c = rows_of(SpanCase(dev, ctx, *args, **kw))
    if spoil:
        c.spoil(window, sinks)
    c.upload()
    live = np.flatnonzero(c.ctx > 0)
    full_q = c.q
    c.q = full_q[torch.from_numpy(live)]
    want = c.expect(window, sinks)
    c.q = full_q
    return c, live, want


def verify(c, live, want, got):
    pkv.check()
    dead = [s for s in range(len(c.ctx)) if s not in set(live.tolist())]
    assert (got[dead] == 0).all()
    check(got[torch.from_numpy(live).to(got.device)], *want, c.d, int(c.ctx.max()), c.dtype, bits(c.dtype))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 16), (15, 4), (16, 0), (17, 17), (33, 40), (64, 4), (100, 0),
                                          (255, 31), (ALL, 0), (7, ALL), (0x7fffffff, 0x7fffffff)])
@pytest.mark.parametrize("d,B,dtype", [(128, 16, "f16"), (64, 4, "bf16")])
def test_windows(cuda_device, window, sinks, d, B, dtype):
    c, live, want = decode_case(cuda_device, EDGES, 4, 2, d, B, dtype, window=window, sinks=sinks, seed=window % 97 + sinks % 7)
    verify(c, live, want, decode(c, window, sinks))


@pytest.mark.parametrize("B", [4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(37, 5), (130, 129)])
def test_blocks(cuda_device, B, d, window, sinks):
    c, live, want = decode_case(cuda_device, [700, 129, 40, 5], 2, 2, d, B, "f16", window=window, sinks=sinks, seed=B + d)
    verify(c, live, want, decode(c, window, sinks))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (6, 2), (4, 1), (7, 1), (8, 1), (9, 1), (12, 1), (16, 1), (17, 1),
                                   (32, 1), (50, 2), (40, 40)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_head_groups(cuda_device, H, Hkv, dtype):
    c, live, want = decode_case(cuda_device, [200, 65, 3], H, Hkv, 128 if H % 2 else 64, 16, dtype, window=70, sinks=3, seed=H)
    verify(c, live, want, decode(c, 70, 3))


@pytest.mark.parametrize("ctx,H,Hkv,window,sinks", [
    ([6000], 8, 8, 4096, 4),            # clusters of 16
    ([6000, 5, 0], 4, 2, 3000, 100),    # clusters with CTAs that have no stage
    ([1500] * 20, 8, 2, 1000, 0),       # clusters of 8 or less
    ([40] * 600, 2, 1, 20, 3),          # more CTAs than fit at once
])
@pytest.mark.parametrize("d", [64, 128])
def test_splits(cuda_device, ctx, H, Hkv, window, sinks, d):
    c, live, want = decode_case(cuda_device, ctx, H, Hkv, d, 16, "bf16", window=window, sinks=sinks, seed=len(ctx))
    verify(c, live, want, decode(c, window, sinks))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(cuda_device, scale):
    c = rows_of(SpanCase(cuda_device, [90, 33], 4, 2, 64, 16, "f16", seed=2)).upload()
    verify(c, np.arange(2), c.expect(50, 3, scale), decode(c, 50, 3, scale=scale))


def test_a_window_over_everything_is_plain_decode(cuda_device):
    c = rows_of(SpanCase(cuda_device, [1, 100, 1000], 8, 2, 128, 16, "f16", seed=4)).upload()
    got = decode(c, 1000, 0)
    plain = pkv.paged_attention_decode(torch.empty_like(got), c.qd, c.kc, c.vc, c.t, c.c)
    want = c.expect()
    verify(c, np.arange(3), want, got)
    half = 2.0 ** -11
    # each is off by its own roundings: the plain call's probabilities carry 11 bits
    assert ((got - plain).abs().double().cpu().numpy() <= 2 * half * np.abs(want[0]) + 3 * half * want[1]).all()


def test_infinite_and_nan_inputs(cuda_device):
    """A NaN query gives NaN rows; -inf scores everywhere give zeros; neither touches other sequences."""
    c = rows_of(SpanCase(cuda_device, [60, 60, 60], 2, 2, 64, 16, "f16", seed=5)).upload()
    clean = decode(c, 40, 2).clone()
    c.qd[0, 0, 3] = math.nan
    c.qd[1] = 0.0
    c.qd[1, :, 0] = 1.0
    blocks = c.t[1].long()
    c.kc[blocks[blocks >= 0], :, :, 0] = -math.inf
    got = decode(c, 40, 2)
    pkv.check()
    assert got[0, 0].isnan().all() and torch.equal(got[0, 1], clean[0, 1])
    assert (got[1] == 0).all() and torch.equal(got[2], clean[2])


def test_a_cache_past_32_bit_offsets(cuda_device):
    """Blocks behind 2^32 elements of a pool."""
    c, live, want = decode_case(cuda_device, [300, 77], 4, 2, 128, 16, "f16", window=100, sinks=4,
                                offset=(1 << 32) // (2 * 16 * 128) + 3)
    verify(c, live, want, decode(c, 100, 4))
    c = SpanCase(cuda_device, [300, 77], 4, 2, 128, 16, "f16", new=[200, 77], seed=9,
                 offset=(1 << 32) // (2 * 16 * 128) + 3).upload()
    pkv.paged_attention_prefill_window(c.out, c.qd, c.kc, c.vc, c.t, c.c, c.qs, 100, 4)
    pkv.check()
    check(c.out, *c.expect(100, 4), c.d, 300, "f16", 11)


def test_bad_blocks_and_contexts_are_latched(cuda_device):
    c = rows_of(SpanCase(cuda_device, [100, 50], 2, 2, 64, 16, "f16", seed=6)).upload()
    good = decode(c, 60, 4).clone()
    pkv.check()
    t = c.t.clone()
    t[0, 5] = c.NB + 7                                  # inside the window
    with pytest.raises(pkv.PkvError, match="block-table entry"):
        pkv.paged_attention_decode_window(c.out, c.qd, c.kc, c.vc, t, c.c, 60, 4)
        pkv.check()
    assert torch.equal(c.out[1], good[1])
    t = c.t.clone()
    t[0, 2] = c.NB + 7                                  # between sinks and window: not read
    pkv.paged_attention_decode_window(c.out, c.qd, c.kc, c.vc, t, c.c, 50, 4)
    pkv.check()
    for bad in (-1, 1 << 20):
        ctx = c.c.clone()
        ctx[0] = bad
        with pytest.raises(pkv.PkvError, match="context length"):
            pkv.paged_attention_decode_window(c.out, c.qd, c.kc, c.vc, c.t, ctx, 60, 4)
            pkv.check()
    assert torch.equal(decode(c, 60, 4), good)


def test_rows_behind_the_batch_stay_and_replays_agree(cuda_device):
    """Captured on a stream, replayed with other inputs, beside eager calls on another stream."""
    c = rows_of(SpanCase(cuda_device, [400, 90, 2000], 8, 2, 128, 16, "bf16", seed=7)).upload()
    big = torch.full((5, 8, 128), 7.0, dtype=torch.bfloat16, device=cuda_device)
    want = decode(c, 300, 4).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_attention_decode_window(big[:3], c.qd, c.kc, c.vc, c.t, c.c, 300, 4)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    eager = torch.empty_like(want)
    for _ in range(3):
        big[:3] = 0
        graph.replay()
        decode(c, 300, 4, out=eager, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(big[:3], want) and torch.equal(eager, want) and (big[3:] == 7).all()
    c.c.copy_(torch.tensor([10, 89, 1000], dtype=torch.int32))
    graph.replay()
    assert torch.equal(big[:3], decode(c, 300, 4))
    pkv.check()


# -- prompts ---------------------------------------------------------------------------

def prompt(c, window, sinks, **kw):
    out = torch.full_like(c.qd, math.nan)
    pkv.paged_attention_prefill_window(out, c.qd, c.kc, c.vc, c.t, c.c, c.qs, window, sinks, **kw)
    pkv.check()
    return out


def prompt_bits(dtype):
    return 11 if dtype == "f16" else 16


def blocks_unseen(c, window, sinks):
    """Entries of blocks that no row sees out of range, and NaN in those blocks."""
    for s in range(len(c.ctx)):
        n, r = int(c.ctx[s]), int(c.new[s])
        low = max(0, n - r - window + 1)
        for j in range(-(-n // c.B)):
            if (j + 1) * c.B <= low and j * c.B >= sinks:
                for x in c.pools:
                    x[c.tables[s, j]] = math.nan
                c.tables[s, j] = (-1, 1 << 30)[j % 2]
    return c


PROMPTS = [  # (contexts, new tokens)
    ([1, 2, 17, 77], [1, 2, 17, 77]),
    ([128, 129, 255, 256, 257], [128, 129, 255, 256, 257]),
    ([640, 500], [640, 130]),
    ([1000, 900, 64], [3, 300, 0]),
    ([1200], [520]),
]


@pytest.mark.parametrize("ctx,new", PROMPTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (32, 4), (127, 0), (128, 129), (129, 4), (300, 16), (513, 200),
                                          (ALL, 0), (9, ALL)])
@pytest.mark.parametrize("H,Hkv,d,B,dtype", [(2, 2, 128, 16, "f16"), (4, 2, 64, 8, "bf16")])
def test_prompts(cuda_device, ctx, new, window, sinks, H, Hkv, d, B, dtype):
    c = blocks_unseen(SpanCase(cuda_device, ctx, H, Hkv, d, B, dtype, new=new, seed=len(ctx) + window % 31), window, sinks)
    c.upload()
    check(prompt(c, window, sinks), *c.expect(window, sinks), d, max(ctx), dtype, prompt_bits(dtype))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (8, 1)])
@pytest.mark.parametrize("B", [4, 32, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_shapes(cuda_device, H, Hkv, B, dtype, d):
    c = blocks_unseen(SpanCase(cuda_device, [700, 330], H, Hkv, d, B, dtype, new=[410, 330], seed=H + B), 150, 20).upload()
    want = c.expect(150, 20)
    check(prompt(c, 150, 20), *want, d, 700, dtype, prompt_bits(dtype))
    ws = pkv.make_workspace(cuda_device, 256)
    for _ in range(2):                                   # the counter is ready again
        check(prompt(c, 150, 20, workspace=ws), *want, d, 700, dtype, prompt_bits(dtype))


@pytest.mark.parametrize("sinks", [1, 4, 15, 16, 17, 33, 64, 100, 127, 129, 150])
@pytest.mark.parametrize("H,Hkv,B,dtype,d", [(2, 2, 16, "f16", 128), (4, 2, 4, "bf16", 64), (1, 1, 128, "f16", 64), (2, 1, 64, "bf16", 128)])
def test_what_lies_behind_the_sinks_has_no_effect(cuda_device, sinks, H, Hkv, B, dtype, d):
    """NaN from the last sink up to well before the first row's window, in the sinks' own blocks too."""
    c = SpanCase(cuda_device, [1000, 1130], H, Hkv, d, B, dtype, new=[300, 90], seed=sinks)
    window = 200
    for s in range(2):
        low = int(c.ctx[s]) - int(c.new[s]) - window + 1
        for t in range(sinks, low - 127):
            for x in c.pools:
                x[c.tables[s, t // B], :, t % B] = math.nan
    c = blocks_unseen(c, window, sinks).upload()
    check(prompt(c, window, sinks), *c.expect(window, sinks), d, 1130, dtype, prompt_bits(dtype))


@pytest.mark.parametrize("S", [1, 33, 70])
def test_prompts_of_many_lengths(cuda_device, S):
    """More sequences than a warp looks at in one go, some without new tokens."""
    rng = np.random.default_rng(S)
    new = rng.integers(0, 300, S) * (rng.random(S) < 0.8)
    new[0] = max(1, new[0])
    ctx = new + rng.integers(0, 200, S)
    for H, Hkv in ((1, 1), (2, 1)):
        c = SpanCase(cuda_device, np.maximum(ctx, 1), H, Hkv, 64, 16, "f16", new=new, seed=S).upload()
        want = c.expect(90, 20)
        check(prompt(c, 90, 20), *want, 64, 500, "f16", 11)
        check(prompt(c, 90, 20, max_query_len=299, workspace=pkv.make_workspace(cuda_device, 256)), *want, 64, 500, "f16", 11)


def test_prompt_rows_are_single_tokens(cuda_device):
    """Every row of a prompt is the decode of its own context."""
    c = SpanCase(cuda_device, [300], 4, 2, 128, 16, "bf16", new=[300], seed=8).upload()
    got = prompt(c, 60, 4)
    ctx = torch.arange(1, 301, dtype=torch.int32, device=cuda_device)
    one = torch.empty_like(got)
    pkv.paged_attention_decode_window(one, c.qd, c.kc, c.vc, c.t.expand(300, -1).contiguous(), ctx, 60, 4)
    pkv.check()
    want = c.expect(60, 4)
    check(got, *want, 128, 300, "bf16", 16)
    check(one, *want, 128, 300, "bf16", 16)


def test_prompt_errors_are_latched(cuda_device):
    c = SpanCase(cuda_device, [300, 64], 2, 2, 64, 16, "f16", new=[40, 64], seed=8).upload()
    t = c.t.clone()
    t[0, 17] = -5                                        # seen
    with pytest.raises(pkv.PkvError, match="block-table entry"):
        pkv.paged_attention_prefill_window(c.out, c.qd, c.kc, c.vc, t, c.c, c.qs, 60, 4)
        pkv.check()
    ctx = c.c.clone()
    ctx[1] = 63                                          # fewer tokens than new ones
    with pytest.raises(pkv.PkvError, match="context length"):
        pkv.paged_attention_prefill_window(c.out, c.qd, c.kc, c.vc, c.t, ctx, c.qs, 60, 4)
        pkv.check()
