"""Arguments of the 8-bit calls at the ends of their ranges (CPU: nothing is launched)."""
import pytest

from test_fp8_host import P, _append, _message, _prefill

NO_DEVICE = 4           # PKV_ECUDA: the arguments were taken, and there is no GPU here to launch on


def _without_a_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that nothing stands behind")


@pytest.mark.parametrize("over", [dict(dt=0, scale=2.0e38), dict(dt=0, scale=3.4e38), dict(dt=1, scale=float("inf"))])
def test_prefill_refuses_scales_that_it_cannot_double(over):
    """fp16 keys are widened at half their size, with twice the scale."""
    assert _prefill(**over) == 1 and "scale" in _message()


def test_prefill_takes_the_largest_scales():
    _without_a_gpu()
    assert _prefill(dt=0, scale=1.7e38) == NO_DEVICE and _prefill(dt=1, scale=3.4e38) == NO_DEVICE


@pytest.mark.parametrize("over", [dict(S=1000, T=1 << 20, H=4096, Hkv=1), dict(S=65535, T=1 << 20, H=129, Hkv=1),
                                  dict(S=60000, T=2 ** 31 - 1, mql=12800, H=360, Hkv=2)])
def test_prefill_refuses_too_many_work_items_before_it_widens(over):
    """What the prompt-phase kernel would refuse is refused before anything is launched."""
    assert _prefill(wsb=1 << 50, **over) == 1 and "work items" in _message() and "prefill_fp8" in _message()


def test_prefill_takes_as_many_work_items_as_the_kernel():
    _without_a_gpu()
    sizes = dict(T=1 << 23, mql=256 * 256, H=256, Hkv=256, wsb=1 << 50)                 # 2^16 items a sequence
    assert _prefill(S=(1 << 14) - 1, **sizes) == NO_DEVICE and _prefill(S=1 << 14, **sizes) == 1


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refuses_to_rotate_strided_queries_in_place(fp8):
    """query_out is contiguous: its rows would lie over other tokens' queries that are still to be read."""
    assert _append(fp8, qs=768) == 1 and "in place" in _message()
    _without_a_gpu()
    assert _append(fp8, qs=768, qo=2 * P) == NO_DEVICE and _append(fp8, qs=768, T=1) == NO_DEVICE
    assert _append(fp8) == NO_DEVICE


def test_workspaces_hold_the_partitions_that_the_kernels_make():
    """The kernels take partitions of 2^30 tokens at most: contexts past that are two, whatever size was asked for."""
    import paged_kv_cache_139_gb300 as pkv
    size = pkv.paged_attention_workspace_size
    n = 2 ** 31 - 1
    for P in (1 << 30, 2 ** 31 - 32):
        assert size(1, 1, 1, 64, n, P) == size(1, 1, 1, 64, 600, 512) > 256
        assert size(1, 1, 1, 64, 1 << 30, P) == 256
    assert size(1, 1, 1, 64, 2 ** 31 - 64, 2 ** 31 - 32) == size(1, 1, 1, 64, 600, 512)
    assert size(3, 4, 2, 64, 1000, 2 ** 31 - 32) == size(3, 4, 2, 64, 1000, 1024) == 256
    size8 = pkv.paged_attention_decode_fp8_workspace_size
    assert size8(3, 4, 2, 64, 1000, 2 ** 31 - 64) == size8(3, 4, 2, 64, 1000, 1024) == 256
