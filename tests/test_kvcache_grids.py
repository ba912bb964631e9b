"""Every launch of an attention call that is accepted has fewer than 2^32 threads a dimension (HIP
refuses others), also with the default max_q = tokens in front of many sequences (no GPU needed)."""
import random

import pytest

import kv_plan
from scale_search_weights_amd import kvcache
from test_abi import ESHAPE, FAKE
from test_kvcache_host import C, attention

LOOSE = [
    # dtype, tokens, heads, batch, max_q, max_kv, prefix, kv_heads, head_dim
    (1, 8192, 32, 8192, 8192, 2000, 0, 8, 128),      # 2^23 workgroups of 512 threads
    (1, 8192, 32, 8192, 8192, 2000, 900, 8, 128),
    (0, 8192, 32, 8192, 8192, 2000, 900, 8, 256),
    (1, 65535, 4, 65535, 65535, 100, 0, 4, 64),
    (1, 65535, 1024, 65535, 1, 100, 0, 1024, 64),    # exact bounds: 2^26 workgroups of 256 threads
]


def covered(sizes):
    p, ls = kv_plan.plan(*sizes), kv_plan.launches(*sizes)
    assert all(1 <= g and g * t < 1 << 32 for _, _, g, t in ls)
    for k, r in enumerate((p.prefix, p.own)):
        mine = [l for l in ls if l[0] == k]
        units = sizes[7] * r.row_tiles
        both = k == 1 and r.slots and not mine  # in the prefix's launch
        if both:
            one, = (l for l in ls if l[0] == 0)
            assert one[2] == units * r.slots + sizes[7] * p.prefix.row_tiles * p.prefix.slots
            continue
        at = 0
        for n, (_, first, g, t) in enumerate(mine):
            assert first == at and t == 64 * r.waves
            if n + 1 < len(mine) or k == 1:
                assert g % units == 0
                at += g // units
        assert k == 0 or at == r.slots
    return ls


@pytest.mark.parametrize("sizes", LOOSE)
def test_loose_bounds_are_launched_in_turns(sizes):
    assert kv_plan.plan(*sizes).fits
    assert len(covered(sizes)) > 1


def test_any_call():
    rng = random.Random(1)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    for _ in range(4000):
        kv_heads, batch = rng.choice((1, 2, 8, 64, 1024)), log(1, 65535)
        heads, max_q = kv_heads * rng.choice((1, 2, 4, 16)), log(1, 100000)
        tokens = min(max_q * batch, log(max_q, 10 * max_q))
        if tokens * heads > (1 << 31) - 1024:
            continue
        sizes = (rng.randint(0, 1), tokens, heads, batch, max_q, rng.choice((0, log(1, 1 << 20))),
                 rng.choice((0, log(1, 1 << 20))), kv_heads, rng.choice((16, 64, 96, 128, 256)))
        if kv_plan.plan(*sizes).fits:
            covered(sizes)


def test_what_cannot_be_launched_is_refused():
    """More than 2^31 workgroups, and a join of 2^32 threads."""
    sizes = (1, 65535, 512, 65535, 65535, 2000, 0, 32, 128)
    assert not kv_plan.plan(*sizes).fits
    c = dict(kv_heads=32, head_dim=128)
    kw = dict(tokens=65535, heads=512, ts=65536, hs=128, batch=65535, offs=FAKE, max_q=65535)
    L = kvcache.lib()
    assert attention(L, C(**c), **kw) == ESHAPE
    assert L.nvfp4_kv_attention_workspace_size(C(**c), 1, 65535, 512, 65535, 65535, 4096, 0) == 0
    kw = dict(tokens=1 << 21, heads=32, ts=8192, hs=256, batch=1, max_q=1 << 21, prefix=5000, pp=FAKE)
    assert attention(L, C(head_dim=256), **kw) == ESHAPE
