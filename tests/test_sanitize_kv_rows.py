"""The rows of a sequence, computed as the kernels do, under UndefinedBehaviorSanitizer (no GPU
needed)."""
import os

from test_sanitize import HERE, _run


def test_rows_of_a_sequence_in_32_bits(tmp_path):
    exe = str(tmp_path / "kv_rows_checks")
    _run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=all",
          os.path.join(HERE, "kv_rows_checks.cpp"), "-o", exe])
    assert "kv rows checks passed" in _run([exe], sanitized=True).stdout
