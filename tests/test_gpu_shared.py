"""Decode over shared prefixes on the GPU against 64 bits: groups of one row to
several tiles of them, prefixes of any length, splits of both halves."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from span_reference import SpanCase, check

pytestmark = pytest.mark.gpu


def shared(c, out=None, **kw):
    out = torch.full_like(c.qd, math.nan) if out is None else out
    return pkv.paged_attention_decode_shared(out, c.qd, c.kc, c.vc, c.t, c.c, c.gs, c.pl, **kw)


def bounds(c):
    return dict(max_context_len=int(c.ctx.max()), max_prefix_len=int(c.prefix.max()), max_group_size=max(c.groups),
                max_suffix_len=int((c.ctx - c.prefix).max()))


def p_bits(c):
    few = max(c.groups) * (c.H // c.Hkv) <= 16
    return 16 if c.dtype == "bf16" else 22 if few else 11


def make(dev, groups, prefix, suffix, *args, seed=0, **kw):
    rng = np.random.default_rng(seed)
    ctx = np.repeat(prefix, groups) + (rng.integers(suffix[0], suffix[1] + 1, sum(groups)))
    return SpanCase(dev, ctx, *args, groups=groups, prefix=prefix, seed=seed, new=np.ones(len(ctx), np.int64), **kw)


def verify(c, got):
    pkv.check()
    check(got, *c.expect(), c.d, int(c.ctx.max()), c.dtype, p_bits(c))


@pytest.mark.parametrize("groups,prefix,suffix", [
    ([1], [16], (1, 1)),
    ([3], [100], (0, 9)),                                # no own token at all
    ([4, 1, 2], [0, 33, 128], (1, 40)),                  # a group without a prefix
    ([2, 2], [500, 129], (1, 300)),
    ([40], [300], (1, 20)),
    ([70, 5], [257, 1], (0, 65)),
    ([130, 1, 33], [1000, 128, 127], (1, 17)),
])
@pytest.mark.parametrize("H,Hkv,d,B,dtype", [(2, 2, 128, 16, "f16"), (4, 1, 64, 8, "bf16"), (4, 2, 128, 32, "bf16"),
                                             (12, 2, 64, 16, "f16")])
def test_groups(cuda_device, groups, prefix, suffix, H, Hkv, d, B, dtype):
    # (a prefix and no own token: the sequences of a group see the same tokens; without either there is no context)
    if 0 in prefix and suffix[0] == 0:
        suffix = (1, suffix[1])
    c = make(cuda_device, groups, prefix, suffix, H, Hkv, d, B, dtype, seed=len(groups) + H).upload()
    verify(c, shared(c, **bounds(c)))


def wide(c, tokens=1 << 17):
    """The same tables with room for many more tokens, so that a call without bounds takes the prefixes for long
    ones: larger groups then go through the prompt phase's kernel."""
    c.t = torch.nn.functional.pad(c.t, (0, tokens // c.B - c.t.shape[1]), value=-1).contiguous()
    return c


@pytest.mark.parametrize("groups,prefix,suffix", [
    ([17], [16], (1, 1)),
    ([30], [100], (0, 9)),
    ([40, 1, 2], [300, 33, 128], (1, 40)),
    ([70, 5], [257, 1], (0, 65)),
    ([64, 20], [0, 512], (1, 300)),
    ([130, 1, 33], [1000, 128, 127], (1, 17)),
])
@pytest.mark.parametrize("H,Hkv,d,B,dtype", [(2, 2, 128, 16, "f16"), (4, 1, 64, 8, "bf16"), (4, 2, 128, 32, "bf16"),
                                             (14, 2, 64, 16, "f16"), (1, 1, 128, 128, "f16")])
def test_large_groups(cuda_device, groups, prefix, suffix, H, Hkv, d, B, dtype):
    if 0 in prefix and suffix[0] == 0:
        suffix = (1, suffix[1])
    c = wide(make(cuda_device, groups, prefix, suffix, H, Hkv, d, B, dtype, seed=len(groups) + H).upload())
    verify(c, shared(c))
    verify(c, shared(c, max_group_size=max(groups), max_suffix_len=int((c.ctx - c.prefix).max())))


@pytest.mark.parametrize("groups,prefix,H,Hkv", [([64], [4000], 8, 4), ([40, 9], [3000, 100], 12, 4), ([300], [700], 8, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_groups_in_partitions(cuda_device, groups, prefix, H, Hkv, dtype, d):
    c = make(cuda_device, groups, prefix, (1, 1300), H, Hkv, d, 16, dtype, seed=len(groups) + 1).upload()
    verify(c, shared(c, **bounds(c)))


@pytest.mark.parametrize("B", [4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("n", [2, 20])
def test_blocks(cuda_device, B, n):
    c = make(cuda_device, [n, 3], [390, 200], (1, 60), 4, 4, 128, B, "f16", seed=B).upload()
    verify(c, shared(c, **bounds(c)))
    verify(c, shared(c))                                 # without bounds


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (7, 1), (16, 1), (17, 1), (100, 1), (128, 1), (24, 2)])
@pytest.mark.parametrize("n", [1, 5, 37])
def test_head_groups(cuda_device, H, Hkv, n):
    c = make(cuda_device, [n, 2], [260, 64], (1, 20), H, Hkv, 64 if H % 2 else 128, 16, "bf16", seed=H).upload()
    verify(c, shared(c, **bounds(c)))
    verify(c, shared(wide(c)))


@pytest.mark.parametrize("groups,prefix,suffix,H,Hkv", [
    ([64], [4000], (1, 30), 4, 2),                       # a prefix in many partitions
    ([3], [6000], (1, 3000), 2, 2),                      # own tokens in clusters
    ([2] * 150, [64] * 150, (1, 8), 4, 4),               # more groups than fit at once
    ([300], [700], (1, 8), 8, 2),                        # many row tiles
])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_splits(cuda_device, groups, prefix, suffix, H, Hkv, dtype):
    c = make(cuda_device, groups, prefix, suffix, H, Hkv, 128, 16, dtype, seed=len(groups)).upload()
    verify(c, shared(c, **bounds(c)))


def test_empty_contexts_and_empty_batches(cuda_device):
    c = make(cuda_device, [2, 2], [0, 48], (1, 5), 4, 2, 64, 16, "f16").upload()
    c.c[0] = 0
    got = shared(c, **bounds(c))
    pkv.check()
    assert (got[0] == 0).all()
    want, mag, x = c.expect()
    check(got[1:], want[1:], mag[1:], x, 64, 60, "f16", 22)
    none = torch.empty(0, 4, 64, dtype=torch.float16, device=cuda_device)
    i = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    pkv.paged_attention_decode_shared(none, none, c.kc, c.vc, i.view(0, 1), i, i.new_zeros(1), i)
    pkv.check()


def test_agrees_with_plain_decode(cuda_device):
    c = make(cuda_device, [6, 30], [200, 331], (1, 50), 8, 2, 128, 16, "bf16", seed=3).upload()
    plain = pkv.paged_attention_decode(torch.empty_like(c.out), c.qd, c.kc, c.vc, c.t, c.c)
    got = shared(c, **bounds(c))
    want = c.expect()
    verify(c, got)
    half = 2.0 ** -8
    assert ((got - plain).abs().double().cpu().numpy() <= 2 * half * np.abs(want[0]) + 3 * half * want[1]).all()


@pytest.mark.parametrize("n", [4, 40])
def test_only_the_first_sequences_table_is_read_for_the_prefix(cuda_device, n):
    c = make(cuda_device, [n], [160], (1, 50), 4, 2, 64, 16, "f16", seed=5).upload()
    c.t[1:, :10] = 1 << 30
    verify(c, shared(c, **bounds(c)))
    verify(c, shared(wide(c)))


@pytest.mark.parametrize("n,far", [(2, False), (30, False), (30, True)])
def test_bad_groups_are_latched(cuda_device, n, far):
    c = make(cuda_device, [n, 2], [100, 40], (1, 30), 4, 2, 64, 16, "f16", seed=6).upload()
    kw = bounds(c)
    if far:                                              # through the prompt phase's kernel
        wide(c)
        kw = dict(max_group_size=n)
    good = shared(c, **kw).clone()
    pkv.check()

    def refused(match, gs=None, pl=None, ctx=None, t=None, **over):
        with pytest.raises(pkv.PkvError, match=match):
            pkv.paged_attention_decode_shared(torch.empty_like(good), c.qd, c.kc, c.vc, c.t if t is None else t,
                                              c.c if ctx is None else ctx, c.gs if gs is None else gs,
                                              c.pl if pl is None else pl, **{**kw, **over})
            pkv.check()

    at = lambda x, i, v: x.index_fill(0, torch.tensor([i], device=x.device), v)  # noqa: E731
    refused("group of sequences", gs=at(c.gs, 0, 1))
    refused("group of sequences", gs=at(c.gs, 2, n + 1))
    refused("group of sequences", gs=at(c.gs, 1, n + 9))
    refused("group of sequences", gs=at(c.gs, 1, -4))
    refused("group of sequences", pl=at(c.pl, 1, 99))
    refused("group of sequences", max_group_size=n - 1)
    refused("context length", pl=at(at(c.pl, n, 1000), n + 1, 1000))
    refused("context length", pl=c.pl.index_fill(0, torch.arange(n, n + 2, device=c.pl.device), -3))
    refused("context length", ctx=at(c.c, 0, 99))
    refused("context length", max_prefix_len=64, max_context_len=0 if far else kw["max_context_len"])
    bad = c.t.clone()
    bad[0, 3] = -1
    refused("block-table entry", t=bad)
    bad = c.t.clone()
    bad[1, 6] = c.NB
    refused("block-table entry", t=bad)
    assert torch.equal(shared(c, **kw), good)
    pkv.check()


@pytest.mark.parametrize("n,prefix", [(3, 300), (50, 300), (50, 2700)])
def test_captured_steps_and_streams(cuda_device, n, prefix):
    """Two captured graphs and an eager stream, each with memory of its own, and one workspace for calls in turn."""
    c = make(cuda_device, [n, 2], [prefix, 64], (1, 40), 8, 2, 128, 16, "f16", seed=7).upload()
    kw = bounds(c)
    want = shared(c, **kw).clone()
    outs = [torch.zeros_like(want) for _ in range(3)]
    graphs = []
    for o in outs[:2]:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            shared(c, out=o, **kw)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for o in outs:
            o.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        shared(c, out=outs[2], stream=streams[2], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    size = pkv.paged_attention_decode_shared_workspace_size(len(c.ctx), 2, 8, 2, 128, **kw)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=cuda_device)           # NaN, whatever is read before it is written
    for _ in range(3):
        assert torch.equal(shared(c, workspace=ws, **kw), want)
    with pytest.raises(pkv.PkvError, match="workspace"):
        shared(c, workspace=ws[:-16], **kw)
    pkv.check()


def test_a_wrong_guess_of_the_own_tokens_changes_nothing(cuda_device):
    for groups, far in (([3, 2], False), ([40, 2], False), ([40, 2], True)):
        c = make(cuda_device, groups, [130, 60], (1, 3000), 4, 2, 64, 16, "bf16", seed=12).upload()
        kw = dict(max_group_size=40) if far else bounds(c)
        if far:
            wide(c)
        for guess in (1, 17, 300, 0):
            verify(c, shared(c, **{**kw, "max_suffix_len": guess}))


def test_a_cache_past_32_bit_offsets(cuda_device):
    c = make(cuda_device, [20], [100], (1, 30), 4, 2, 128, 16, "f16", offset=(1 << 32) // (2 * 16 * 128) + 3).upload()
    verify(c, shared(c, **bounds(c)))
    verify(c, shared(wide(c)))
