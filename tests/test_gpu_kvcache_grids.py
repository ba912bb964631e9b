"""Attention calls whose workgroups do not fit one launch."""
import pytest
import torch

import kvcache_ref as ref
import kv_plan
from scale_search_weights_amd import kvcache
from test_gpu_kvcache import BF, DEV, case, check, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 40])
def test_many_sequences_behind_the_default_max_q(prefix):
    """8192 sequences of one query, max_q left at 8192: launched in turns, all rows are written."""
    n, heads, kv_heads, hd = 8192, 32, 8, 64
    case(f"kv attention, {n} sequences, max_q = tokens, prefix {prefix}")
    lens = [(7 * b) % 45 for b in range(n)]
    own = [l for l in kv_plan.launches(1, n, heads, n, n, 48, prefix, kv_heads, hd) if l[0] == 1]
    assert len(own) > 1
    c = ref.make(n, BF, [1] * n, lens, heads, kv_heads, hd, 16, prefix)
    cache, q, table, kv_lens = on_gpu(c), c["q"].contiguous().to(DEV), c["table"].to(DEV), c["kv_lens"].to(DEV)
    pages = c["prefix_pages"].to(DEV) if prefix else None
    got = []
    for bound in (None, 1):
        out = torch.full(q.shape, float("nan"), dtype=BF, device=DEV)
        got.append(kvcache.attention(cache, q, table, kv_lens, q_offsets=c["q_offsets"].to(DEV), max_q=bound, max_kv=48,
                                     prefix_pages=pages, prefix_len=prefix, out=out, return_lse=True))
    # either is within A (2^-11 + ..) + |out| 2^-8 of the truth, A <= max |v| <= 6 * 64 * S_v
    far = (got[0][0].float() - got[1][0].float()).abs().max().item()
    assert far <= 2.0 ** -6 * 6 * 64 * float(c["cache"][5].max())
    at = torch.tensor([0, 1, 2, 4000, first(own), first(own) - 1, n - 1])
    sub = dict(c, q=c["q"][at], table=c["table"][at], kv_lens=c["kv_lens"][at], q_offsets=torch.arange(len(at) + 1))
    for out, lse in got:
        check(sub, (out[at.to(DEV)], lse[at.to(DEV)]))


def first(launches):
    """The first sequence of the second launch."""
    return launches[1][1]
