"""Rotations and appends of the sizes at which workgroups take several tokens, rows pass the dies' caches or
heads fall into several groups. test_rotary_variants.py holds the lists to that with the host plan,
test_gpu_rotary_variants.py runs them."""
import ctypes
import functools
import os
import subprocess
import tempfile
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
BF16, FP32 = 1, 0
Turn = namedtuple("Turn", "dtype tokens heads hd pairs axes adjacent factor")
Append = namedtuple("Append", "dtype tokens heads kv_heads hd pairs page axes adjacent factor")
Rows = namedtuple("Rows", "units heads groups")
TurnPlan = namedtuple("TurnPlan", "v tokens rows stream")
AppendPlan = namedtuple("AppendPlan", "tokens kv q stream")

# pieces of 8 and 4 values, halves and adjacent pairs, stored past the caches and left in them; the tokens are
# no multiple of what a workgroup takes
TURNS = [
    Turn(BF16, 12001, 32, 128, 64, 3, False, 1.0), Turn(BF16, 9003, 32, 128, 64, 1, True, 1.2),
    Turn(FP32, 9801, 16, 72, 36, 2, False, 1.0), Turn(FP32, 11003, 10, 80, 24, 1, True, 1.0),
    Turn(BF16, 20003, 13, 72, 36, 2, False, 1.0), Turn(BF16, 14001, 16, 88, 20, 3, True, 0.75),
    Turn(BF16, 16383, 3, 64, 32, 2, False, 1.0), Turn(BF16, 5003, 5, 64, 16, 1, True, 1.0),
    Turn(FP32, 7001, 2, 24, 12, 1, False, 1.0), Turn(FP32, 4099, 4, 40, 12, 2, True, 1.0),
    Turn(BF16, 30001, 1, 8, 4, 1, False, 1.0), Turn(BF16, 6007, 3, 24, 12, 1, True, 1.0)]

APPENDS = [
    # several groups of heads in every role, the last one smaller
    Append(BF16, 48, 40, 40, 128, 64, 16, 1, False, 1.0), Append(BF16, 9, 70, 70, 64, 32, 16, 3, False, 1.0),
    Append(FP32, 5, 19, 9, 1024, 512, 16, 1, False, 1.0), Append(BF16, 13, 141, 47, 96, 24, 32, 2, True, 1.25),
    Append(FP32, 7, 75, 75, 32, 8, 16, 1, True, 1.0), Append(BF16, 4001, 70, 70, 16, 8, 64, 1, False, 1.0),
    # several tokens a workgroup, queries past the caches and within them
    Append(BF16, 4511, 32, 8, 128, 64, 64, 3, False, 1.0), Append(BF16, 6007, 28, 4, 128, 40, 64, 1, True, 1.2),
    Append(FP32, 5501, 20, 5, 80, 24, 32, 1, False, 1.0), Append(FP32, 4507, 16, 2, 128, 64, 16, 2, True, 1.0),
    Append(BF16, 3001, 7, 1, 64, 32, 128, 2, True, 1.0), Append(FP32, 2503, 3, 1, 48, 16, 16, 1, False, 1.0),
    Append(BF16, 8003, 0, 1, 32, 16, 64, 1, False, 1.0)]


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "rotary_variants.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC",
                        os.path.join(HERE, "native", "rotary_variants.cpp"), "-o", out], check=True)
        return ctypes.CDLL(out)


def turn_plan(c):
    o = (ctypes.c_int64 * 6)()
    lib().rotary_turn((ctypes.c_int64 * 5)(*c[:5]), o)
    return TurnPlan(o[0], o[1], Rows(*o[2:5]), bool(o[5]))


def append_plan(c):
    o = (ctypes.c_int64 * 8)()
    lib().rotary_append((ctypes.c_int64 * 6)(*c[:6]), o)
    return AppendPlan(o[0], Rows(*o[1:4]), Rows(*o[4:7]), bool(o[7]))
