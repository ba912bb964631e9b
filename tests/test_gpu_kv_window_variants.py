"""Every kernel variant of windowed attention, whole and in pieces, against 64 bits (the cases are
kv_window_cases.py's, the bounds kv_window_ref.py's)."""
import pytest

import kv_window_cases
import kv_window_ref as win
import kvcache_ref as ref
from test_gpu_kv_window import BF, F32, attend, case

pytestmark = pytest.mark.gpu
CASES = kv_window_cases.cases()


@pytest.mark.parametrize("c", CASES, ids=[f"{i}-{c.what.replace(', ', '-').replace(' ', '_')}" for i, c in enumerate(CASES)])
def test_variant(c):
    case(f"kv window, {c.what}")
    x = ref.make(c.hd + len(c.q_lens) + c.window, BF if c.dtype else F32, c.q_lens, c.kv_lens, c.heads, c.kv_heads, c.hd, 32)
    win.check(x, attend(x, c.window, c.sinks), c.window, c.sinks)
