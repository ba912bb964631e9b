"""The decoding example end to end: write, read and attention as they are used together. The bounds
are the format's: with block scales within a factor of two of the block's maximum a random normal
value is off by about a tenth (relative norm), a softmax over many tokens averages the values'
share of that, and the keys' share moves the scores by about a tenth of their spread."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_example():
    print("[case] decoding example: 5 users, 700-token prompt, 70 steps", flush=True)
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import kv_decode
    r = kv_decode.run(users=5, prompt=700, steps=70)
    assert r["bytes_per_value"] == 0.5625
    assert 0.01 < r["key_error"] < 0.2
    assert 0.0 < r["output_error"] < 0.4
    assert torch.isfinite(r["prompt_out"].float()).all() and torch.isfinite(r["out"].float()).all()
    again = kv_decode.run(users=5, prompt=700, steps=70)
    assert torch.equal(again["prompt_out"], r["prompt_out"]) and torch.equal(again["out"], r["out"])
