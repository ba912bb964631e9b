"""Calls that reach every kernel variant and plan of the cache's attention; test_kvcache_variants.py
holds the list to that with the host plan, test_gpu_kvcache_variants.py runs it."""
from collections import namedtuple

BF16, FP32 = 1, 0
Case = namedtuple("Case", "what dtype q_lens kv_lens heads kv_heads hd prefix causal hidden")
HEAD_DIMS = ((64, 48, 16), (128, 96), (256, 160, 240))  # of each kernel size: the size itself, and some below it


def _ragged(n, most, seed):
    """Lengths from 0 to most, the first most, the second 0."""
    x = [(seed + 7919 * (b + 1) * (b + 3)) % (most + 1) for b in range(n)]
    return [most, 0][:n] + x[2:]


def _case(what, dtype, q_lens, kv_lens, heads, kv_heads, hd, prefix=0, causal=True, hidden=()):
    return Case(f"{what}, {'bf16' if dtype else 'fp32'}, head_dim {hd}", dtype, q_lens, kv_lens, heads, kv_heads, hd,
                prefix, causal, hidden)


def cases():
    out = []
    for size, pair in zip((64, 128, 256), HEAD_DIMS):
        for hd in pair:
            for dtype in (BF16, FP32):
                # many rows: 64 sequences of 8 heads, so that the tiles need not be small
                for q, group in ((33, 1), (33, 2), (65, 2)):
                    q_lens = [q, 0, 1] + [1 + (5 * b) % q for b in range(61)]
                    kv = [max(n, k) for n, k in zip(q_lens, _ragged(64, 90, hd + q))]
                    out.append(_case(f"{q * group} rows", dtype, q_lens, kv, 8 * group, 8, hd, causal=q != 65))
                # up to 16 and up to 32 rows, whole and in pieces
                out.append(_case("20 rows", dtype, [5, 0, 1, 3], [300, 9, 0, 77], 8, 2, hd))
                out.append(_case("20 rows in pieces", dtype, [5, 2], [2700, 900], 8, 2, hd))
                out.append(_case("6 rows in pieces", dtype, [2, 0, 1], [2000, 40, 1999], 6, 2, hd))
                # a prefix in the same launch, and one of many rows in front of pieces
                out.append(_case("short prefix", dtype, [1, 2, 1], [100, 0, 31], 8, 2, hd, 70, hidden=(2,)))
                out.append(_case("short prefix, own tokens in pieces", dtype, [1, 2, 1], [200, 0, 131], 8, 2, hd, 70))
                out.append(_case("long prefix, own tokens in pieces", dtype, [8, 8, 7], [2500, 0, 700], 16, 8, hd, 5600))
                # sequences that fill tiles go over the prefix first; a prefix alone, at once and in pieces
                out.append(_case("prefix first", dtype, [64, 60, 0], [64, 90, 100], 4, 2, hd, 60, hidden=(1,)))
                out.append(_case("prefix alone", dtype, [3, 1], [0, 0], 4, 2, hd, 100))
                out.append(_case("prefix alone in pieces", dtype, [30, 11], [0, 0], 8, 2, hd, 700, hidden=(0, 9)))
            if size == 256:
                continue
            # contexts whole, bf16: 16, 8 and 4 waves a workgroup, alone and finishing a prefix's pieces
            for waves, batch, kv_heads, group, prefix in ((16, 16, 8, 4, 2100), (8, 40, 8, 4, 1700), (4, 70, 8, 3, 1400)):
                kv = _ragged(batch, 260, hd + waves)
                out.append(_case(f"whole, {waves} waves", BF16, [1] * batch, kv, kv_heads * group, kv_heads, hd))
                q_lens = [1 + b % 4 for b in range(batch)]
                q_lens[2:4] = [0, 4]
                own = [max(n, k) if k else 0 for n, k in zip(q_lens, kv)]
                out.append(_case(f"prefix finished, {waves} waves", BF16, q_lens, own, kv_heads * group, kv_heads, hd,
                                 prefix, hidden=(3, 40)))
    return out


def sizes(c):
    """Arguments of kv_plan.plan."""
    return (c.dtype, sum(c.q_lens), c.heads, len(c.q_lens), max(c.q_lens), max(c.kv_lens), c.prefix, c.kv_heads, c.hd)
