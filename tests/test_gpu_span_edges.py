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
