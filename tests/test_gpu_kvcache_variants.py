"""Every kernel variant and plan of the cache's attention against the 64-bit reference, with the bounds
of test_gpu_kvcache.py (the cases are kv_cases.py's)."""
import pytest

import kv_cases
import kvcache_ref as ref
from test_gpu_kvcache import BF, F32, attend, case, check

pytestmark = pytest.mark.gpu
CASES = kv_cases.cases()


@pytest.mark.parametrize("c", CASES, ids=[f"{i}-{c.what.replace(', ', '-').replace(' ', '_')}" for i, c in enumerate(CASES)])
def test_variant(c):
    case(f"kv attention, {c.what}")
    x = ref.make(c.hd + len(c.q_lens) + c.prefix, BF if c.dtype else F32, c.q_lens, c.kv_lens, c.heads, c.kv_heads, c.hd, 16,
                 c.prefix)
    for n, page in enumerate(c.hidden):
        x["prefix_pages"][page] = (-1, 1 << 20)[n % 2]
    check(x, attend(x, causal=c.causal), c.causal)
