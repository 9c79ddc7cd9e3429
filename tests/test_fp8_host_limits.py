"""Arguments of the 8-bit calls at the ends of their ranges (CPU: nothing is launched)."""
import pytest

from test_fp8_host import _message, _prefill

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
