"""Rotary and 8-bit calls at the edges of what their definitions allow."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import F8, RefCache8, rotate32
from test_gpu_rotary import DT, Inputs, _random_cache8, _same8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rot,layout", [(64, 0, "half"), (128, 0, "half"), (128, 32, "half"), (64, 48, "interleaved"),
                                          (128, 128, "half"), (64, 64, "interleaved")])
@pytest.mark.parametrize("B", [4, 16, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append8_nan_rows_do_not_count(cuda_device, dtype, B, d, rot, layout):
    """Whole rows of NaN among the tokens that one call writes to a block: scales and the other rows' codes are those of
    the numbers alone, in blocks begun anew and in partly filled ones, also where nothing but NaN is written."""
    H, Hkv, NB = 2, 3, 12
    # block 0 anew, 1 and 2 from their second row, 3 anew and all NaN, 4 partly filled and all NaN, 5 and 6 one token each
    slots = np.concatenate([np.arange(B), B + 1 + np.arange(B - 1), 2 * B + 1 + np.arange(2), 3 * B + np.arange(B),
                            4 * B + 2 + np.arange(2), [5 * B, 6 * B + 3]]).astype(np.int64)
    T = len(slots)
    x = Inputs(cuda_device, T, H, Hkv, d, B, dtype, B + d, rot, NB=NB, strided=False)
    block = slots // B
    k, v = x.k.clone(), x.v.clone()
    k[1], v[0] = math.nan, math.nan                             # whole tokens
    k[B, 1], v[B + 1, 2], k[B + 2, 0, :32] = math.nan, math.nan, math.nan       # a head's row; the first part of one
    v[torch.from_numpy(block == 2)] = math.nan
    for b in (3, 4):
        k[torch.from_numpy(block == b)] = v[torch.from_numpy(block == b)] = math.nan
    k[-1] = v[-2] = math.nan
    k0, v0, s0 = _random_cache8(NB, Hkv, B, d, B)
    kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
    dk, dv = k.to(cuda_device), v.to(cuda_device)
    args = (x.dq, dk, dv, x.dcs, x.dpos) if rot else (None, dk, dv, None, None)
    pkv.kv_rotary_and_cache_fp8(*args, kc, vc, sc, torch.from_numpy(slots).to(cuda_device), layout=layout)
    pkv.check()
    ref = RefCache8(k0, v0, s0)
    ref.append(rotate32(k, x.cs, x.positions, rot, layout).numpy(), v.float().numpy(), slots)
    _same8(ref, kc, vc, sc, "NaN rows")
