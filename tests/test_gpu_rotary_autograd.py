"""The rotation under autograd's hooks and modes, on the GPU (tests/test_rotary_autograd.py: the host path)."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from scale_search_weights_amd import rotary

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _make(dtype=torch.bfloat16):
    gen = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(77, 5, 96, generator=gen, device=DEV).to(dtype)
    pos = torch.randint(0, 5000, (3, 77), generator=gen, device=DEV)
    return x, pos, rotary.Rotary.create(96, sections=(8, 20, 20), factor=1.25)


def test_activations_kept_on_the_host():
    print("[case] rotate backward with saved tensors on the host", flush=True)
    x, pos, rot = _make()
    g = torch.randn_like(x)
    want = rotary.rotate(g, pos, rot, transpose=True)
    with torch.autograd.graph.save_on_cpu():
        y = rotary.rotate(x.clone().requires_grad_(), pos, rot)
    leaf = y.grad_fn.next_functions[0][0].variable
    rot.inv_freq.mul_(1.5)  # torch compares no versions here: the copies count
    rot.axis.copy_(2 - rot.axis)
    pos.add_(3)
    y.backward(g)
    assert torch.equal(leaf.grad, want)


def test_forward_mode_and_followed_outputs_are_refused():
    print("[case] rotate: forward mode and outputs in a graph", flush=True)
    x, pos, rot = _make(torch.float32)
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            rotary.rotate(forward_ad.make_dual(x, torch.ones_like(x)), pos, rot)
    a = torch.randn_like(x).requires_grad_()
    with pytest.raises(ValueError):
        rotary.rotate(x, pos, rot, out=a * 2)
    with torch.no_grad():
        assert torch.equal(rotary.rotate(x, pos, rot, out=a), rotary.rotate(x, pos, rot))
