"""How rotation and append are split into workgroups (csrc/nvfp4_rotary_plan.h): every row once, within
LDS, 16-bit item numbers and the threads that a launch takes (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
TABLE, HEADS = 2048, 64
TOKENS = (1, 2, 7, 48, 511, 16384, 12345677, (1 << 31) - 1)


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "rotary_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "native", "rotary_plan.cpp"),
                    "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.rotary_launches.restype = ctypes.c_int64
    return lib


def _launches(L, tokens, n, groups):
    out = (ctypes.c_int64 * 40000)()
    k = L.rotary_launches(ctypes.c_int64(tokens), n, ctypes.c_int64(groups), out, ctypes.c_int64(20000))
    assert k <= 20000
    return [(out[2 * i], out[2 * i + 1]) for i in range(k)]


def _covers(launches, tokens, n):
    at = 0
    for chunks, t0 in launches:
        assert t0 == at
        at += chunks * n
    assert at >= tokens > at - n


@pytest.mark.parametrize("bf16", [0, 1])
@pytest.mark.parametrize("hd,pairs", [(8, 4), (72, 36), (80, 20), (128, 64), (1016, 508), (1024, 512), (1024, 4)])
def test_rotate(L, bf16, hd, pairs):
    for tokens in TOKENS:
        for heads in (1, 3, 32, 65535):
            o = (ctypes.c_int64 * 5)()
            L.rotary_rotate_plan(bf16, ctypes.c_int64(tokens), ctypes.c_int64(heads), ctypes.c_int64(hd), pairs, o)
            v, n, units, per, groups = o
            assert pairs % v == 0 and hd % (2 * v) == 0 and 2 * v * units == hd
            assert n >= 1 and n * pairs <= TABLE and n * per * units < 1 << 16
            assert 1 <= per <= heads and groups * per >= heads > (groups - 1) * per and groups <= 65535
            if tokens < 1 << 30 or n > 1:
                ls = _launches(L, tokens, n, groups)
                _covers(ls, tokens, n)
                assert all(c * 256 < 1 << 32 for c, _ in ls)


@pytest.mark.parametrize("bf16", [0, 1])
@pytest.mark.parametrize("hd,pairs", [(16, 8), (80, 40), (96, 24), (128, 64), (1024, 512), (1024, 8)])
def test_append(L, bf16, hd, pairs):
    for tokens in TOKENS:
        for heads, kv_heads in ((0, 1), (32, 8), (7, 7), (65535, 1), (0, 65535), (1000, 1000)):
            o = (ctypes.c_int64 * 7)()
            L.rotary_append_plan(bf16, ctypes.c_int64(tokens), ctypes.c_int64(heads), ctypes.c_int64(kv_heads),
                                 ctypes.c_int64(hd), pairs, o)
            n, units, per, groups, q_units, q_per, q_groups = o
            assert 16 * units == hd and q_units == (units if bf16 else 2 * units)
            assert n >= 1 and n * pairs <= TABLE and n * per * units < 1 << 16 and n * q_per * q_units < 1 << 16
            assert 1 <= per <= min(kv_heads, HEADS) and groups * per >= kv_heads > (groups - 1) * per
            assert q_per >= 1 and q_groups * q_per >= heads > (q_groups - 1) * q_per
            every = 2 * groups + q_groups
            if tokens < 1 << 26:
                ls = _launches(L, tokens, n, every)
                _covers(ls, tokens, n)
                # chunks are dealt to eight dies, so their number is rounded up
                assert all((c + 7) // 8 * 8 * every * 256 < 1 << 32 for c, _ in ls)


def test_quotients_by_multiplication():
    """The kernels' n / d = (n m) >> 32 with m = 2^32 // d + 1, for every n below 2^16 and many d."""
    for d in [*range(2, 300), 511, 512, 513, 1000, 4095, 4096, 32767, 65535]:
        m = (1 << 32) // d + 1
        assert m < 1 << 32
        for n in [*range(0, 1 << 16, 97), *range(0, 1 << 16, d), *range(d - 1, 1 << 16, d), (1 << 16) - 1]:
            assert n * m >> 32 == n // d
