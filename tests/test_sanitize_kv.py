"""The key/value cache's host code under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU
needed), built and run as test_sanitize.py does for the other entry points."""
import os
import subprocess

from scale_search_weights_amd import build as hip_build
from test_sanitize import HERE, SAN_HOST, _run

SOURCES = ["nvfp4_kv.hip", "nvfp4_kv_attn.hip", "nvfp4_kv_api.hip", "nvfp4_debug.hip"]


def test_kv_host_code_under_sanitizers(tmp_path):
    common = [*hip_build.FLAGS, *SAN_HOST, "-Xarch_host", "-g", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs, procs = [], []
    for src in [*(os.path.join(hip_build.CSRC, s) for s in SOURCES), os.path.join(HERE, "kv_checks.cpp")]:
        objs.append(str(tmp_path / (os.path.basename(src).split(".")[0] + ".o")))
        procs.append(subprocess.Popen([hip_build.HIPCC, *common, "-c", src, "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.PIPE))
    for p in procs:
        _, err = p.communicate()
        assert p.returncode == 0, err.decode()[-3000:]
    exe = str(tmp_path / "kv_checks")
    _run([hip_build.HIPCC, *SAN_HOST, *objs, "-o", exe])
    assert "kv checks passed" in _run([exe], sanitized=True).stdout
