"""Queries that are not finite: their rows come out as NaN (out and lse) whatever the plan (one
piece written directly, pieces joined, a prefix in the same launch, apart or first, many rows, heads
of every kernel size), rows that see nothing stay 0 and -inf, and every other row is right."""
import math

import pytest
import torch

import kvcache_ref as ref
from test_gpu_kvcache import BF, F32, attend, case, check

pytestmark = pytest.mark.gpu

PLANS = [
    # dtype, q_lens, kv_lens, heads, kv_heads, hd, prefix
    ("whole", BF, [1, 1], [900, 33], 8, 2, 128, 0),
    ("pieces", BF, [1, 1], [9000, 200], 8, 2, 128, 0),
    ("pieces fp32", F32, [1, 2], [700, 300], 8, 2, 128, 0),
    ("pieces wide", BF, [1], [1500], 4, 1, 256, 0),
    ("prefix in the same launch", BF, [1] * 3, [30, 0, 200], 8, 2, 128, 60),
    ("prefix finished by the own tokens", BF, [1] * 64, [70] * 63 + [0], 16, 4, 64, 2100),
    ("prefix and own tokens joined", BF, [20, 3], [90, 300], 8, 2, 128, 3000),
    ("many rows", BF, [150], [260], 4, 2, 128, 0),
    ("many rows in pieces", BF, [40], [2600], 2, 1, 64, 0),
    ("many rows fp32", F32, [80], [130], 4, 2, 128, 0),
    ("prefix first", BF, [128, 100], [128, 110], 4, 2, 128, 77),
    ("prefix alone", BF, [2, 1], [0, 0], 8, 2, 128, 500),
]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("what,dtype,q_lens,kv_lens,heads,kv_heads,hd,prefix", PLANS, ids=[p[0] for p in PLANS])
def test_queries_that_are_not_finite(what, dtype, q_lens, kv_lens, heads, kv_heads, hd, prefix, bad):
    case(f"kv attention, {bad} in a query, {what}")
    c = ref.make(len(q_lens) + hd, dtype, q_lens, kv_lens, heads, kv_heads, hd, 16, prefix)
    good = attend(c)
    spots = {(0, 0, 0), (c["q"].shape[0] - 1, heads - 1, hd - 1), (c["q"].shape[0] // 2, heads // 2, hd // 2)}
    q = c["q"].clone()
    rows = torch.zeros(q.shape[:2], dtype=torch.bool)
    for t, h, d in spots:
        q[t, h, d] = bad
        rows[t, h] = True
    out, lse = attend(dict(c, q=q))
    empty = torch.isneginf(good[1].cpu())
    assert rows.any() and not (rows & ~empty).sum() == 0
    nan = (rows & ~empty).to(out.device)
    assert torch.isnan(out[nan].float()).all() and torch.isnan(lse[nan]).all()
    blank = (rows & empty).to(out.device)
    assert (out[blank] == 0).all() and torch.isneginf(lse[blank]).all()
    out[nan], lse[nan] = good[0][nan], good[1][nan]
    check(c, (out, lse))
