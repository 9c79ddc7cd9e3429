"""Windowed and shared-prefix attention on the GPU where limits meet: windows and
sinks at the ends of 32 bits, edges at every offset of a box and block."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from span_reference import SpanCase, check

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("window,sinks", [(MOST, 0), (MOST - 1, 4), (MOST - 100, MOST), (1 << 30, MOST), (5, MOST), (5, MOST - 127)])
@pytest.mark.parametrize("H,Hkv,d,B,dtype", [(2, 2, 128, 16, "f16"), (4, 2, 64, 8, "bf16")])
def test_prompts_at_the_ends_of_32_bits(cuda_device, window, sinks, H, Hkv, d, B, dtype):
    c = SpanCase(cuda_device, [700, 257, 300], H, Hkv, d, B, dtype, new=[700, 129, 1], seed=window % 13).upload()
    pkv.paged_attention_prefill_window(c.out, c.qd, c.kc, c.vc, c.t, c.c, c.qs, window, sinks)
    pkv.check()
    check(c.out, *c.expect(window, sinks), d, 700, dtype, 11 if dtype == "f16" else 16)


# At head_dim 128, blocks of more than four tokens and more items than fit at once, the stages that hold a limit of
# what is seen come in boxes of four tokens.  480 items of one to 90 tokens.

def many(dev, B, dtype, seed, **kw):
    rng = np.random.default_rng(seed)
    return SpanCase(dev, rng.integers(1, 91, 120), 8, 4, 128, B, dtype, seed=seed, **kw)


@pytest.mark.parametrize("B", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (6, 1), (19, 3), (33, 18), (50, 6)])
def test_edges_of_windows_in_many_items(cuda_device, B, dtype, window, sinks):
    c = many(cuda_device, B, dtype, window + B).spoil(window, sinks).upload()
    pkv.paged_attention_decode_window(c.out, c.qd, c.kc, c.vc, c.t, c.c, window, sinks)
    pkv.check()
    check(c.out, *c.expect(window, sinks), 128, 90, dtype, 22 if dtype == "f16" else 16)


@pytest.mark.parametrize("B", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("groups,large", [([3] * 40, False), ([20, 17, 23, 60], True)])
def test_edges_of_own_tokens_in_many_items(cuda_device, B, dtype, groups, large):
    rng = np.random.default_rng(B + len(groups))
    prefix = rng.integers(0, 70, len(groups))
    ctx = np.repeat(prefix, groups) + rng.integers(1, 41, sum(groups))
    c = SpanCase(cuda_device, ctx, 8, 4, 128, B, dtype, groups=groups, prefix=prefix, new=np.ones(len(ctx), np.int64), seed=B)
    c.upload()
    if large:          # room for long prefixes, so that the prompt phase's kernel takes them
        c.t = torch.nn.functional.pad(c.t, (0, (1 << 15) // B - c.t.shape[1]), value=-1).contiguous()
    n = pkv.launch_count()
    pkv.paged_attention_decode_shared(c.out, c.qd, c.kc, c.vc, c.t, c.c, c.gs, c.pl, max_suffix_len=40,
                                      max_group_size=max(groups), max_prefix_len=0 if large else int(prefix.max()))
    assert pkv.launch_count() - n == (3 if large else 2)
    pkv.check()
    check(c.out, *c.expect(), 128, int(ctx.max()), dtype, 16 if dtype == "bf16" else 11 if large else 22)
