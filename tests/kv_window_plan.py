"""The host plan of windowed attention (csrc/nvfp4_kv_window_plan.h), compiled for the tests."""
import ctypes
import functools
import os
import subprocess
import tempfile
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
Plan = namedtuple("Plan", "fits nt waves tile row_tiles slots pieces direct workspace")


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "kv_window_plan.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC",
                        os.path.join(HERE, "native", "kv_window_plan.cpp"), "-o", out], check=True)
        return ctypes.CDLL(out)


def plan(*sizes):
    """Of (dtype, tokens, heads, batch, max_q, max_kv, window, sinks, kv_heads, head_dim)."""
    out = (ctypes.c_int64 * 8)()
    fits = _lib().kv_window_plan((ctypes.c_int64 * 10)(*sizes), out)
    return Plan(bool(fits), *out)


def launches(*sizes):
    """(list, first slot, workgroups, threads of one) of every launch."""
    out = (ctypes.c_int64 * 4096)()
    n = _lib().kv_window_launches((ctypes.c_int64 * 10)(*sizes), out, 1024)
    assert n <= 1024
    return [tuple(out[4 * i:4 * i + 4]) for i in range(n)]
