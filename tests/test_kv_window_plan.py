"""The host plan of windowed attention: the cases of kv_window_cases.py reach every kernel variant that is
built, whole and in pieces; sizes at their extremes; launches within what HIP takes (no GPU needed)."""
import pytest

import kv_window_cases
import kv_window_plan
from kv_window_cases import BF16, FP32


def built():
    """What launch_rows has for a window's calls: (size, exact, dtype, tile, 16-row tiles, waves)."""
    out = set()
    for size in (64, 128, 256):
        for dtype in (BF16, FP32):
            wide, f32 = size == 256, dtype == FP32
            rows = [(1, 4)] + ([] if wide and f32 else [(2, 4)]) + ([] if wide or f32 else [(1, 8)])
            tile = [(1, 4)] + ([(1, 8)] if wide != f32 else [] if wide else [(2, 4), (2, 8)])
            for exact in (True, False):
                out |= {(size, exact, dtype, 0, *x) for x in rows} | {(size, exact, dtype, 1, *x) for x in tile}
    return out


def test_every_variant_whole_and_in_pieces():
    seen = set()
    for c in kv_window_cases.cases():
        p = kv_window_plan.plan(*kv_window_cases.sizes(c))
        size = 64 if c.hd <= 64 else 128 if c.hd <= 128 else 256
        assert p.fits and p.direct == (p.pieces == 1) and (p.workspace == 0) == (p.pieces == 1)
        seen.add((size, c.hd == size, c.dtype, p.tile, p.nt, p.waves, p.pieces > 1))
    want = {(*v, cut) for v in built() for cut in (False, True)}
    assert len(built()) == 52  # full attention has 56, four of them with sixteen waves
    assert seen == want, (want - seen, seen - want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("hd", [16, 64, 80, 128, 256])
def test_extremes(dtype, hd):
    big = 1 << 30
    for heads, kvh in ((1, 1), (64, 8), (65535, 65535)):
        for batch, tokens, max_q in ((1, 1, 1), (65535, 65535, 1), (1, 32, 32), (1, 33, 33), (1, 30000, 30000),
                                     (65535, 30000, 30000), (1, 2 ** 31 - 1025, 2 ** 31 - 1025)):
            if tokens * heads > 2 ** 31 - 1025:
                continue
            for max_kv in (0, 1, 127, 100000, big):
                for window, sinks in ((1, 0), (1, big), (big, 0), (big, big), (4096, 128)):
                    s = (dtype, tokens, heads, batch, max_q, max_kv, window, sinks, kvh, hd)
                    p = kv_window_plan.plan(*s)
                    assert p.nt >= 1 and p.waves in (4, 8) and p.pieces >= 1 and p.slots == batch * p.pieces
                    rows = max_q * (heads // kvh)
                    tile = 16 * p.nt * (p.waves if p.tile else 1)
                    assert p.row_tiles * tile >= rows > (p.row_tiles - 1) * tile
                    if p.pieces > 1:
                        # partial sums of a few rounds of the chip at most, however long the context
                        assert p.slots * kvh * p.row_tiles <= 1024 + 256 and p.workspace > 0
                    if not p.fits:
                        continue
                    if batch * p.pieces * kvh * p.row_tiles < 1 << 26:
                        ls = kv_window_plan.launches(*s)
                        assert all(g * t < 1 << 32 for _, _, g, t in ls)
                        assert sum(g for k, _, g, _ in ls if k != 2) == p.slots * kvh * p.row_tiles
                        assert (ls[-1][0] == 2) == (p.pieces > 1)


def test_work_does_not_grow_with_the_context():
    for q in (1, 8, 40, 2000):
        a, b = (kv_window_plan.plan(BF16, q, 32, 1, q, n, 1024, 4, 8, 128) for n in (20000, 1 << 30))
        assert a == b
