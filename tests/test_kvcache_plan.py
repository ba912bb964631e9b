"""How the attention's host plan splits a call (no GPU needed)."""
import pytest

from scale_search_weights_amd import kvcache
from test_kvcache_host import C


def workspace(batch, max_kv, heads, kv_heads, hd, dtype=1, max_q=1, prefix=0):
    c = C(head_dim=hd, kv_heads=kv_heads)
    return kvcache.lib().nvfp4_kv_attention_workspace_size(c, dtype, batch * max_q, heads, batch, max_q, max_kv, prefix)


@pytest.mark.parametrize("batch,max_kv,heads,kv_heads,hd,cut", [
    # us a call cut and whole, launched one by one | from a graph
    (1, 400, 32, 8, 128, False),    # 12.3, 9.8 | 9.9, 9.5
    (4, 1000, 32, 8, 128, False),   # 12.7, 11.6 | 10.6, 11.7
    (4, 1500, 32, 8, 128, True),    # 12.6, 14.1 | 12.2, 14.1
    (1, 1500, 8, 1, 128, True),     # graph 10.7, 14.5
    (2, 1500, 32, 8, 96, True),     # 12.8, 16.9 | 11.7, 16.9
    (5, 1500, 32, 8, 128, True),    # 12.7, 14.0 | 12.4, 14.1
    (7, 1500, 32, 8, 128, False),   # graph 13.6, 13.9; at 1200 tokens 13.4, 12.6
    (10, 1000, 32, 8, 128, False),  # graph 13.2, 12.0
    (1, 1500, 20, 20, 64, False),   # 12.7, 11.3 | 10.4, 11.1
    (1, 2000, 20, 20, 64, True),    # at 1900 tokens 12.7, 12.0 | 11.2, 11.7
    (5, 1500, 20, 20, 64, False),   # 13.1, 11.3 | 13.1, 11.4
    (30, 6000, 32, 8, 128, False),  # graph 43.0, 37.8
])
def test_contexts_are_cut_where_both_ways_of_calling_are_faster_for_it(batch, max_kv, heads, kv_heads, hd, cut):
    """A context cut into pieces needs a workspace for their sums, a whole one does not."""
    assert (workspace(batch, max_kv, heads, kv_heads, hd) > 0) == cut
