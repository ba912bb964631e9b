"""The attention's host plan (csrc/nvfp4_kv_plan.h), compiled for the tests."""
import ctypes
import functools
import os
import subprocess
import tempfile
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
Part = namedtuple("Part", "nt waves tile row_tiles slots")
Plan = namedtuple("Plan", "fits prefix own cut direct finish lead")
JOIN = 2  # the list number of the join's launch


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "kv_plan.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "native", "kv_plan.cpp"),
                        "-o", out], check=True)
        return ctypes.CDLL(out)


def _sizes(dtype, tokens, heads, batch, max_q, max_kv, prefix, kv_heads, hd):
    return (ctypes.c_int64 * 9)(dtype, tokens, heads, batch, max_q, max_kv, prefix, kv_heads, hd)


def plan(*sizes):
    """Of (dtype, tokens, heads, batch, max_q, max_kv, prefix_len, kv_heads, head_dim)."""
    out = (ctypes.c_int64 * 14)()
    fits = _lib().kv_plan(_sizes(*sizes), out)
    return Plan(bool(fits), Part(*out[0:5]), Part(*out[5:10]), *(bool(x) for x in out[10:14]))


def launches(*sizes):
    """(list, first slot, workgroups, threads of one) of every launch."""
    out = (ctypes.c_int64 * 4096)()
    n = _lib().kv_launches(_sizes(*sizes), out, 1024)
    assert n <= 1024
    return [tuple(out[4 * i:4 * i + 4]) for i in range(n)]
