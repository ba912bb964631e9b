"""Calls that reach every kernel variant of windowed attention, whole and in pieces; test_kv_window_plan.py
holds the list to that with the host plan, test_gpu_kv_window_variants.py runs it."""
from collections import namedtuple

BF16, FP32 = 1, 0
Case = namedtuple("Case", "what dtype q_lens kv_lens heads kv_heads hd window sinks")
HEAD_DIMS = ((64, 64), (64, 48), (128, 128), (128, 96), (256, 256), (256, 160))  # kernel size, head_dim
# (sequences, query tokens, key/value heads, query heads of each, window) by type and kernel size
SHAPES = {
    (BF16, 64): [(1, 1, 1, 1, 16), (1, 1, 1, 1, 2000), (1, 1, 1, 1, 300), (40, 1, 2, 1, 2000), (1, 5, 1, 4, 16),
                 (1, 5, 1, 4, 900), (1, 33, 1, 1, 16), (1, 60, 1, 1, 300), (40, 60, 8, 4, 16), (40, 20, 2, 4, 2000),
                 (8, 130, 8, 4, 900), (8, 130, 8, 1, 2000)],
    (BF16, 128): [(1, 1, 1, 1, 16), (1, 1, 1, 1, 2000), (1, 1, 1, 1, 300), (40, 1, 2, 1, 2000), (1, 5, 1, 4, 16),
                  (1, 5, 1, 4, 900), (1, 33, 1, 1, 16), (1, 33, 1, 1, 300), (40, 20, 8, 4, 100), (4, 130, 8, 4, 2000),
                  (8, 130, 8, 4, 16), (8, 33, 8, 4, 2000)],
    (BF16, 256): [(1, 1, 1, 1, 16), (1, 1, 1, 1, 900), (1, 5, 1, 4, 16), (1, 5, 1, 4, 900), (1, 33, 1, 1, 16),
                  (1, 33, 1, 1, 300), (40, 20, 8, 4, 16), (4, 33, 8, 4, 900)],
    (FP32, 64): [(1, 1, 1, 1, 16), (1, 1, 1, 1, 900), (1, 5, 1, 4, 16), (1, 5, 1, 4, 900), (1, 33, 1, 1, 16),
                 (1, 33, 1, 1, 300), (40, 60, 2, 4, 16), (40, 20, 1, 4, 900)],
    (FP32, 128): [(1, 1, 1, 1, 16), (1, 1, 1, 1, 900), (1, 5, 1, 4, 16), (1, 5, 1, 4, 900), (1, 33, 1, 1, 16),
                  (1, 33, 1, 1, 300), (40, 60, 2, 4, 16), (4, 33, 8, 4, 900)],
    (FP32, 256): [(1, 1, 1, 1, 16), (1, 1, 1, 1, 900), (1, 33, 1, 1, 16), (1, 33, 1, 1, 300)],
}


def cases():
    out = []
    for size, hd in HEAD_DIMS:
        for dtype in (BF16, FP32):
            for n, q, kvh, g, w in SHAPES[dtype, size]:
                # the first sequence is the longest in both; the second is idle, others short and long
                q_lens = [q] + [(0, 1, q, 1 + q // 3)[b % 4] for b in range(n - 1)]
                most = w + q + 30
                kv = [most] + [max(q_lens[b], (0, 17, most - 5, w // 2)[(b - 1) % 4]) for b in range(1, n)]
                out.append(Case(f"{n} x {q} tokens, {g} of {kvh} heads, window {w}, {'bf16' if dtype else 'fp32'}, "
                                f"head_dim {hd}", dtype, q_lens, kv, g * kvh, kvh, hd, w, 4 if q % 2 else 21))
    return out


def sizes(c):
    """Arguments of kv_window_plan.plan."""
    return (c.dtype, sum(c.q_lens), c.heads, len(c.q_lens), max(c.q_lens), max(c.kv_lens), c.window, c.sinks, c.kv_heads,
            c.hd)
