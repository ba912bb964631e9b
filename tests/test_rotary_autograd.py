"""What autograd is told of the rotation: the host path of ``rotate`` with its launch replaced by a plain one (no
GPU needed; test_gpu_rotary.py has the gradients' values)."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import rotary_ref as ref
from scale_search_weights_amd import kvcache, rotary
from test_abi import G, no_launch  # noqa: F401


@pytest.fixture
def plain(monkeypatch):
    """The launch on the CPU, at the frequencies and axes of the Rotary it is given."""
    def launch(x, positions, rot, transpose, out=None):
        turn = ref.turns(positions.as_subclass(torch.Tensor), rot.inv_freq.as_subclass(torch.Tensor), rot.axis, rot.axes)
        with torch.no_grad():
            y = ref.rounded(x.as_subclass(torch.Tensor), turn, rot.adjacent, rot.factor, transpose).to(x.dtype)
            return y if out is None else out.copy_(y)
    monkeypatch.setattr(rotary, "_launch", launch)


def make(tokens=5, heads=2, hd=16):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(tokens, heads, hd, generator=gen)
    pos = torch.randint(0, 1000, (tokens,), generator=gen).as_subclass(type(G(1)))
    w = G(hd // 2, dtype=torch.float64)
    w += 10.0 ** -torch.arange(hd // 2, dtype=torch.float64)
    return x, pos, rotary.Rotary(w)


@pytest.mark.parametrize("grad", [True, False], ids=["gradient mode", "no_grad"])
def test_a_tangent_is_refused_not_dropped(plain, grad):
    """Forward mode is not offered; torch says so, also of a primal that needs no gradient."""
    x, pos, rot = make()
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            rotary.rotate(dual, pos, rot)
        with pytest.raises(ValueError):
            rotary.rotate(dual, pos, rot, out=torch.empty_like(x))
        y = rotary.rotate(x, pos, rot)  # nothing to follow
        assert forward_ad.unpack_dual(y).tangent is None and torch.equal(y, rotary.rotate(x, pos, rot))


def test_a_tangent_of_the_gradient_is_refused_not_dropped(plain):
    x, pos, rot = make()
    y = rotary.rotate(x.requires_grad_(), pos, rot)
    with forward_ad.dual_level():
        g = forward_ad.make_dual(torch.ones_like(x), torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            torch.autograd.grad(y, x, g)


def test_second_order(plain):
    """The gradient is followed where its own input is, and only there."""
    x, pos, rot = make()
    y = rotary.rotate(x.requires_grad_(), pos, rot)
    v, u = torch.randn_like(x).requires_grad_(), torch.randn_like(x)
    gx, = torch.autograd.grad(y, x, v, create_graph=True)
    gv, = torch.autograd.grad(gx, v, u)
    assert torch.equal(gv, rotary.rotate(u, pos, rot))
    y = rotary.rotate(x, pos, rot)
    gx, = torch.autograd.grad(y, x, u, create_graph=True)
    assert not gx.requires_grad and torch.equal(gx, rotary.rotate(u, pos, rot, transpose=True))


def _graph_outputs(shape):
    leaf = G(*shape).requires_grad_()
    return {"a leaf": leaf, "a result": leaf * 2, "a view of a leaf": leaf[:, :, :]}


@pytest.mark.parametrize("kind", ["a leaf", "a result", "a view of a leaf"])
def test_outputs_in_a_graph_are_refused(no_launch, monkeypatch, kind):  # noqa: F811
    """What is overwritten would keep the history of what it held."""
    monkeypatch.setattr(kvcache, "_bound", None)
    monkeypatch.setattr(rotary, "_bound", None)
    _, pos, rot = make()
    out = _graph_outputs((5, 2, 16))[kind]
    x, slots, version = G(5, 2, 16), G(5, dtype=torch.int64), out._version
    cache = kvcache.KVCache(G(4, 2, 16, 8, dtype=torch.uint8), G(4, 2, 16, 1, dtype=torch.uint8),
                            G(4, 2, 16, 8, dtype=torch.uint8), G(4, 2, 16, 1, dtype=torch.uint8), G(2), G(2))
    calls = [lambda: rotary.rotate(x, pos, rot, out=out),
             lambda: kvcache.append(cache, x, x, slots, pos, rot, q=x, q_out=out),
             lambda: kvcache.append(cache, x, x, slots, pos, rot, q=out, q_out=out)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert out._version == version
    with torch.no_grad():  # the caller's own doing, and what autograd saved of it counts as changed
        assert rotary._given_out(out, "out", x) == (32, 16) and out._version == version + 1


def test_outputs_with_a_tangent_are_refused(no_launch, monkeypatch):  # noqa: F811
    monkeypatch.setattr(rotary, "_bound", None)
    _, pos, rot = make()
    with forward_ad.dual_level(), torch.no_grad():
        out = forward_ad.make_dual(G(5, 2, 16), G(5, 2, 16))
        with pytest.raises(ValueError, match="gradient"):
            rotary.rotate(G(5, 2, 16), pos, rot, out=out)


def test_backward_takes_the_frequencies_that_forward_had(plain):
    """Saved-tensor hooks (activations kept on the host, say) hand backward copies, and torch compares no versions
    then: whatever the tensors hold meanwhile, the gradient is the transpose of the turn that was made."""
    x, pos, _ = make()
    w = 10.0 ** -torch.arange(8, dtype=torch.float64) + G(8, dtype=torch.float64)
    axis, at = G(8, dtype=torch.int32), torch.stack((pos, 3 * pos + 1))
    axis[::3] = 1
    rot, before = (rotary.Rotary(a, b, axes=2, factor=1.25) for a, b in ((w, axis), (w.clone(), axis.clone())))
    g = torch.randn_like(x)
    want = rotary.rotate(g, at, rot, transpose=True)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
        y = rotary.rotate(x.requires_grad_(), at, rot)
    w += 1.0
    axis[:] = 1 - axis
    at += 5
    v = g.clone().requires_grad_()
    gx, = torch.autograd.grad(y, x, v, create_graph=True, retain_graph=True)
    assert torch.equal(gx, want)
    gv, = torch.autograd.grad(gx, v, g)
    assert torch.equal(gv, rotary.rotate(g, at - 5, before))


@pytest.mark.parametrize("window", [None, 7])
@pytest.mark.parametrize("kind", ["a leaf", "a result", "a view of a leaf"])
def test_attention_refuses_outputs_in_a_graph(no_launch, monkeypatch, kind, window):  # noqa: F811
    monkeypatch.setattr(kvcache, "_bound", None)
    u8 = torch.uint8
    cache = kvcache.KVCache(G(4, 2, 16, 8, dtype=u8), G(4, 2, 16, 1, dtype=u8), G(4, 2, 16, 8, dtype=u8),
                            G(4, 2, 16, 1, dtype=u8), G(2), G(2))
    out = _graph_outputs((5, 2, 16))[kind]

    def call():
        kvcache.attention(cache, G(5, 2, 16), G(5, 4, dtype=torch.int32), G(5, dtype=torch.int32), window=window, out=out)
    version = out._version
    with pytest.raises(ValueError, match="gradient"):
        call()
    assert out._version == version
    with torch.no_grad(), pytest.raises(AssertionError, match="library"):  # goes on to the launch
        call()
    assert out._version == version + 1
