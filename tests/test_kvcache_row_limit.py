"""Query rows (tokens times heads) whose tiles would pass 32-bit indices are refused (no GPU needed)."""
import pytest

from scale_search_weights_amd import kvcache
from test_abi import ESHAPE, FAKE
from test_kvcache_host import C, attention

MOST = (1 << 31) - 1 - 1024


@pytest.mark.parametrize("tokens,heads", [((1 << 31) - 1, 1), (MOST + 1, 1), ((1 << 30) - 1, 2)])
def test_rows_next_to_the_end_of_32_bits(tokens, heads):
    L = kvcache.lib()
    c = dict(kv_heads=1, head_dim=16)
    assert attention(L, C(**c), tokens=tokens, heads=heads, ts=0, hs=0, batch=1, max_q=tokens, offs=FAKE) == ESHAPE
    assert attention(L, C(**c), tokens=tokens, heads=heads, ts=0, hs=0, batch=1, max_q=1, offs=FAKE) == ESHAPE
    assert L.nvfp4_kv_attention_workspace_size(C(**c), 1, tokens, heads, 1, 1, 4096, 0) == 0


def test_rows_below_that_are_planned():
    L = kvcache.lib()
    assert L.nvfp4_kv_attention_workspace_size(C(kv_heads=1, head_dim=16), 1, MOST, 1, 1, 1, 100000, 0) > 0
