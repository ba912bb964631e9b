"""The cases of rotary_cases.py reach every kernel variant and every shape of a split, and the kernels' quotients
are right (no GPU needed)."""
import ctypes
import itertools

import numpy as np

from rotary_cases import APPENDS, BF16, FP32, TURNS, append_plan, lib, turn_plan


def test_rotations_reach_every_variant():
    plans = [(c, turn_plan(c)) for c in TURNS]
    assert all(p.tokens > 1 and c.tokens % p.tokens for c, p in plans if p.stream or c.heads < 16)
    got = {(c.dtype, p.v, c.adjacent, p.stream) for c, p in plans}
    assert got == set(itertools.product([BF16], [8, 4], [False, True], [False, True])) | \
        set(itertools.product([FP32], [4], [False, True], [False, True]))
    assert {True, False} == {2 * c.pairs < c.hd for c in TURNS} and {1, 2, 3} == {c.axes for c in TURNS}


def test_appends_reach_every_variant():
    plans = [(c, append_plan(c)) for c in APPENDS]
    assert {(c.dtype, c.adjacent, p.stream) for c, p in plans} == \
        set(itertools.product([BF16, FP32], [False, True], [False, True]))
    # several groups of heads, the last one smaller, of both kinds of rows, in both types and kinds of pairs
    uneven = {(c.dtype, c.adjacent) for c, p in plans
              if p.kv.groups > 1 and c.kv_heads % p.kv.heads and p.q.groups > 1 and c.heads % p.q.heads}
    assert uneven == set(itertools.product([BF16, FP32], [False, True])), uneven
    assert any(p.kv.heads == 64 for _, p in plans)  # as many as the scales' table holds
    # several tokens, a last chunk that is not full
    ragged = {(c.dtype, c.adjacent) for c, p in plans if p.tokens > 1 and c.tokens % p.tokens}
    assert ragged == set(itertools.product([BF16, FP32], [False, True])), ragged
    assert any(p.tokens > 1 and p.kv.groups > 1 for _, p in plans) and any(c.heads == 0 for c in APPENDS)


def test_the_kernels_quotients():
    """The code that the kernels run, for every number below 2^16."""
    n, out = np.arange(1 << 16), np.empty(1 << 16, np.int32)
    for d in [*range(1, 1025), *range(1031, 1 << 16, 997), 4095, 4096, 4097, 32767, 32768, 65534, 65535, 65536]:
        lib().rotary_quotients(d, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int)))
        assert np.array_equal(out, n // d), d
