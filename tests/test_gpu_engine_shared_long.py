"""The engine's shared steps over groups large and long enough for the prompt
phase's kernel: direct and prepared, against 64 bits on the CPU."""
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from test_gpu_engine_span import World

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H,Hkv,d,rot", [("bf16", 8, 2, 128, 0), ("f16", 8, 2, 64, 32)])
def test_many_forks_of_a_long_prompt(cuda_device, dtype, H, Hkv, d, rot):
    w = World(cuda_device, dtype, H, Hkv, d, 32, rot=rot)
    a, b = w.eng.new_sequence(0), w.eng.new_sequence(0)
    w.prompt([a, b], [2900, 40])
    batch = [b, a] + [w.fork(a) for _ in range(59)]
    for i in range(3):
        step = w.step(batch, prepared=i == 1, shared=True, few=False)
        assert step.groups.start.tolist() == [0, 1, 61] and step.groups.prefix.tolist() == [0] + [2900 // 32 * 32] * 60
    n = pkv.launch_count()
    w.eng.attend(torch.zeros(61, H, d, dtype=w.eng.key_cache.dtype, device=cuda_device), step)
    assert pkv.launch_count() - n == 3                   # the prefix in the prompt phase's kernel, own tokens, the join
    pkv.check()
