"""Limits of the windowed and shared-prefix calls on the host (no GPU)."""
import pytest

import paged_kv_cache_139_gb300 as pkv
from test_span_host import SHARED, call, message

MANY = dict(S=20000, G=20000, H=16384, Hkv=16384, mgs=17, mpl=128, msl=16, mb=256, wsb=1 << 62)


def test_more_prefix_items_than_the_kernel_can_go_through():
    """20,000 groups x 16,384 kv heads."""
    assert call("paged_attention_decode_shared", SHARED, MANY) == 1
    assert "above 2^27" in message()


@pytest.mark.parametrize("over", [dict(S=-1), dict(G=0), dict(mgs=-1), MANY])
def test_a_refused_call_launches_nothing(over):
    n = pkv.launch_count()
    assert call("paged_attention_decode_shared", SHARED, over) == 1
    assert pkv.launch_count() == n


@pytest.mark.parametrize("name,base,over", [
    ("paged_attention_decode_window", "WINDOW", dict(S=0)), ("paged_attention_prefill_window", "PROMPT", dict(S=0)),
    ("paged_attention_prefill_window", "PROMPT", dict(T=0)), ("paged_attention_decode_shared", "SHARED", dict(S=0, G=0)),
    ("paged_attention_decode_window", "WINDOW", dict(window=0)), ("paged_attention_prefill_window", "PROMPT", dict(scale=0.0))])
def test_calls_with_nothing_to_do_and_refused_ones_launch_nothing(name, base, over):
    import test_span_host
    n = pkv.launch_count()
    assert call(name, getattr(test_span_host, base), over) == (0 if dict(S=0).items() <= over.items() or over == dict(T=0) else 1)
    assert pkv.launch_count() == n
