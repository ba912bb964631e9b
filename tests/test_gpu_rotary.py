"""The rotation on the GPU against its 64-bit definition (tests/rotary_ref.py, which derives the bounds)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import rotary_ref as ref
from scale_search_weights_amd import rotary

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def case(msg):
    print(f"[case] {msg}", flush=True)


def make(seed, dtype, tokens, heads, hd, pairs, axes=1, adjacent=False, factor=1.0, far=200000, base=1e4):
    rng = np.random.default_rng(seed)
    w = torch.from_numpy(base ** (-np.arange(pairs) / pairs))
    axis = torch.from_numpy(rng.integers(0, axes, pairs).astype(np.int32)) if axes > 1 else None
    pos = torch.from_numpy(rng.integers(-far // 8, far, (axes, tokens)))
    # rows of a wider tensor, 8 channels apart where rows stay at multiples of 16 bytes
    x = torch.from_numpy(rng.standard_normal((tokens, heads + 2, hd + 8)).astype(np.float32)).to(dtype)
    rot = rotary.Rotary(w.to(DEV), None if axis is None else axis.to(DEV), axes=axes, adjacent=adjacent, factor=factor)
    return rot, pos, x[:, 1:1 + heads, :hd], ref.turns(pos, w, axis, axes) if far < 1 << 25 else None


def strided(x):
    y = torch.empty(x.shape[0], x.shape[1] + 2, x.shape[2] + 8, dtype=x.dtype, device=DEV)[:, 1:-1, :x.shape[2]]
    y.copy_(x)
    return y


SHAPES = [
    # dtype, tokens, heads, head_dim, pairs, axes, adjacent, factor
    (BF, 1, 1, 8, 4, 1, False, 1.0), (BF, 1, 40, 128, 64, 1, False, 1.0), (F32, 33, 5, 128, 64, 3, False, 1.0),
    (BF, 257, 3, 72, 36, 2, False, 1.0), (F32, 129, 2, 72, 36, 2, True, 1.0), (BF, 70, 7, 80, 20, 1, False, 1.25),
    (BF, 65, 2, 80, 24, 1, True, 0.5), (F32, 31, 3, 80, 40, 1, True, -1.0), (BF, 19, 2, 1024, 512, 1, False, 1.0),
    (F32, 9, 2, 1024, 500, 16, True, 1.0), (BF, 3, 2, 1016, 4, 1, False, 1.0), (BF, 515, 9, 64, 32, 3, True, 1.0),
    (F32, 300, 17, 256, 128, 1, False, 1.1), (BF, 5, 300, 96, 8, 2, False, 1.0), (F32, 17, 2, 24, 12, 1, False, 0.0),
    (BF, 1000, 2, 40, 16, 1, True, 1.0)]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_rotate(shape):
    case(f"rotate {shape}")
    dtype, tokens, heads, hd, pairs, axes, adjacent, factor = shape
    rot, pos, x, turn = make(hd + tokens, *shape[:5], axes, adjacent, factor)
    p = pos[0] if axes == 1 and tokens % 2 else pos
    for transpose in (False, True):
        y = rotary.rotate(strided(x), p.to(DEV), rot, transpose=transpose)
        assert y.dtype == dtype and y.is_contiguous()
        ref.within(y.cpu(), *ref.rotate(x, turn, adjacent, factor, transpose))
        assert torch.equal(y.cpu(), ref.rounded(x, turn, adjacent, factor, transpose).to(dtype))
        assert torch.equal(y[..., 2 * pairs:].cpu(), x[..., 2 * pairs:])


@pytest.mark.parametrize("far,base", [(2 ** 20, 1e4), (2 ** 31, 1e6), (2 ** 40, 1e30)])
def test_far_positions(far, base):
    """Angles up to 2^31 keep their place in the turn: the reference reduces them as fractions."""
    case(f"rotate at positions up to {far}")
    rot, pos, x, _ = make(5, F32, 50, 2, 64, 32, far=far, base=base)
    full = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    theta, keep = torch.zeros(50, 32, dtype=torch.float64), []
    for i, w in enumerate(rot.inv_freq.cpu().tolist()):
        exact = [Fraction(w) * p for p in pos[0].tolist()]
        keep.append(max(map(abs, exact)) <= 2 ** 31)
        if keep[-1]:
            theta[:, i] = torch.tensor([float(a - round(a / full) * full) for a in exact], dtype=torch.float64)
    keep = torch.tensor(keep * 2)
    y = rotary.rotate(strided(x), pos.to(DEV), rot).cpu()
    want, tol = ref.rotate(x, torch.polar(torch.ones_like(theta), theta), False)
    assert keep.sum() >= 8
    ref.within(y[..., keep], want[..., keep], tol[..., keep] + 2.0 ** -48 * x.double().abs().max())
    assert torch.isfinite(y).all()


def test_same_bits_wherever_a_row_stands():
    case("rotate: a row's result does not depend on the others")
    rot, pos, x, _ = make(1, BF, 1025, 33, 128, 64)
    x, pos = strided(x), pos.to(DEV)
    whole = rotary.rotate(x, pos, rot)
    for lo, hi, h0, h1 in ((0, 1, 0, 33), (7, 9, 3, 4), (1000, 1025, 30, 33), (300, 700, 0, 5)):
        assert torch.equal(rotary.rotate(x[lo:hi, h0:h1], pos[:, lo:hi], rot), whole[lo:hi, h0:h1])


def test_layouts_in_place_and_outputs():
    case("rotate: strides, in place, given outputs, broadcast positions")
    rot, pos, x, turn = make(2, F32, 37, 6, 96, 48)
    want = ref.rounded(x, turn, False)
    p = pos.to(DEV)
    y = strided(x)
    out = rotary.rotate(y, p, rot, out=y)
    assert out is y and torch.equal(y.cpu(), want)
    heads_first = x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    assert torch.equal(rotary.rotate(heads_first, p, rot).cpu(), want)
    spare = torch.full((6, 37, 104), 7.0, device=DEV)
    rotary.rotate(heads_first, p, rot, out=spare.transpose(0, 1)[..., :96])
    assert torch.equal(spare.transpose(0, 1)[..., :96].cpu(), want) and (spare[..., 96:] == 7).all()
    # every axis at the same positions, and one token's positions for all
    rot3 = rotary.Rotary(rot.inv_freq, torch.arange(48, device=DEV, dtype=torch.int32) % 3, axes=3)
    assert torch.equal(rotary.rotate(strided(x), p.expand(3, -1), rot3).cpu(), want)
    rows = torch.cat((p, p + 1, p + 2, p + 3))
    assert torch.equal(rotary.rotate(strided(x), rows[::2][:1], rot).cpu(), want)


def test_axis_outside_the_positions_stands_still():
    case("rotate: axes outside the positions")
    rot, pos, x, _ = make(3, F32, 20, 2, 32, 16, axes=2)
    axis = torch.tensor([0, 1, -1, 2, 1 << 30, -(1 << 31)] + [1] * 10, dtype=torch.int32)
    bad = rotary.Rotary(rot.inv_freq, axis.to(DEV), axes=2, factor=1.5)
    turn = ref.turns(pos, rot.inv_freq.cpu(), axis, 2)
    assert torch.equal(rotary.rotate(strided(x), pos.to(DEV), bad).cpu(), ref.rounded(x, turn, False, 1.5))


def test_empty_and_not_finite():
    case("rotate: no rows; values that are not finite stay in their pairs")
    rot, pos, x, turn = make(4, F32, 4, 3, 48, 16)
    for shape in ((0, 3, 48), (4, 0, 48)):
        assert rotary.rotate(torch.empty(shape, device=DEV), pos[:, :shape[0]].to(DEV), rot).shape == shape
    x = x.clone()
    x[1, 2, 5], x[2, 0, 40], x[3, 1, 17] = np.inf, -np.inf, np.nan
    y = rotary.rotate(x.to(DEV), pos.to(DEV), rot).cpu()
    want = ref.rounded(x, turn, False)
    assert torch.equal(torch.isfinite(y), torch.isfinite(want)) and y[2, 0, 40] == -np.inf
    ok = torch.isfinite(want)
    assert torch.equal(y[ok], want[ok])


def test_offsets_past_32_bits():
    case("rotate: rows more than 2^32 bytes apart")
    rot, pos, x, turn = make(6, BF, 3, 2, 64, 32)
    base = torch.empty((1 << 31) * 2 + (1 << 20), dtype=BF, device=DEV)
    y = base.as_strided((3, 2, 64), (1 << 31, 1 << 16, 1))
    y.copy_(x)
    p = pos.to(DEV)
    rotary.rotate(y, p, rot, out=y)
    assert torch.equal(y.cpu(), ref.rounded(x, turn, False).to(BF))
    wide = torch.zeros(2, (1 << 29) + 8, dtype=torch.int64, device=DEV).as_strided((2, 3), ((1 << 29) + 8, 1))
    wide.copy_(pos.expand(2, 3))
    rot2 = rotary.Rotary(rot.inv_freq, torch.ones(32, dtype=torch.int32, device=DEV), axes=2)
    assert torch.equal(rotary.rotate(x.to(DEV), wide, rot2).cpu(), ref.rounded(x, turn, False).to(BF))


# ------------------------------------------------------------------------------------ gradients

@pytest.mark.parametrize("dtype,hd,pairs,adjacent", [(F32, 72, 36, False), (BF, 128, 64, False), (F32, 80, 24, True)])
def test_gradients(dtype, hd, pairs, adjacent):
    case(f"rotate backward {dtype} {hd}/{pairs}")
    rot, pos, x, turn = make(hd, dtype, 45, 4, hd, pairs, axes=2, adjacent=adjacent, factor=1.25)
    g = torch.randn(45, 4, hd, generator=torch.Generator().manual_seed(1)).to(dtype)
    leaf = strided(x).detach().requires_grad_()
    y = rotary.rotate(leaf, pos.to(DEV), rot)
    y.backward(g.to(DEV))
    ref.within(leaf.grad.cpu(), *ref.rotate(g, turn, adjacent, 1.25, True))
    # differences: the map is linear, so (f(x + d) - f(x - d)) / 2 = f(d), and <g, f(d)> = <f^T(g), d>
    d = torch.randn(45, 4, hd, generator=torch.Generator().manual_seed(2)).to(dtype)
    with torch.no_grad():
        up, down = (rotary.rotate(s * d.to(DEV) + leaf.detach(), pos.to(DEV), rot).double() for s in (1, -1))
    moved = ((leaf.detach() + d.to(DEV)).double() - (leaf.detach() - d.to(DEV)).double()) / 2
    left = (g.to(DEV).double() * (up - down) / 2).sum()
    right = (leaf.grad.double() * moved).sum()
    # each side's terms are rounded to the type once (the sums are 64 bits): relative to the sum of magnitudes
    mags = (g.to(DEV).double().abs() * (up.abs() + down.abs())).sum() + (leaf.grad.double().abs() * moved.abs()).sum()
    assert abs(left - right) <= mags * (2.0 ** -8 if dtype == BF else 2.0 ** -21)


def test_gradients_expanded_twice_and_not_asked_for():
    case("rotate backward: expanded gradients, second order, no gradients")
    rot, pos, x, turn = make(8, F32, 21, 3, 64, 32)
    p = pos.to(DEV)
    leaf = strided(x).detach().requires_grad_()
    rotary.rotate(leaf, p, rot).sum().backward()  # the gradient has strides of 0
    assert torch.equal(leaf.grad.cpu(), ref.rounded(torch.ones(21, 3, 64), turn, False, transpose=True))
    odd = torch.randn(21 * 3 * 64 + 1, device=DEV)[1:].view(21, 3, 64)  # contiguous, but off 16 bytes
    gx, = torch.autograd.grad(rotary.rotate(leaf, p, rot), leaf, odd)
    assert torch.equal(gx, rotary.rotate(odd.clone(), p, rot, transpose=True))
    y = rotary.rotate(leaf, p, rot)
    v = torch.randn_like(y).requires_grad_()
    gx, = torch.autograd.grad(y, leaf, v, create_graph=True)
    u = torch.randn_like(y)
    gv, = torch.autograd.grad(gx, v, u)
    assert torch.equal(gv, rotary.rotate(u, p, rot))
    with torch.no_grad():
        assert not rotary.rotate(leaf, p, rot).requires_grad
        rotary.rotate(leaf, p, rot, out=torch.empty_like(y))
    with pytest.raises(ValueError):
        rotary.rotate(leaf, p, rot, out=torch.empty_like(y))
    for changed in (p, rot.inv_freq):  # meanwhile
        y = rotary.rotate(leaf, p, rot)
        changed += 1
        with pytest.raises(RuntimeError):
            y.sum().backward()


# ------------------------------------------------------------------------------ streams and graphs

def test_side_stream_and_graph():
    case("rotate on a side stream and in a graph, forward and backward")
    rot, pos, x, _ = make(9, BF, 500, 6, 128, 64)
    p, a = pos.to(DEV), x.to(DEV)
    want = rotary.rotate(a, p, rot)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rotary.rotate(a, p, rot)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    leaf, g = a.clone().requires_grad_(), torch.randn_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rotary.rotate(leaf, p, rot)
        dx, = torch.autograd.grad(y, leaf, g)
    for step in range(4):
        with torch.no_grad():
            leaf.copy_(a * (step + 1))
            g.copy_(a - step)
        p.add_(step)
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            assert torch.equal(y, rotary.rotate(leaf, p, rot))
            assert torch.equal(dx, rotary.rotate(g, p, rot, transpose=True))


def test_expanded_inputs_and_outputs_that_autograd_saved():
    case("rotate: one row for all heads; a given output that an eager graph saved")
    rot, pos, x, turn = make(10, F32, 30, 1, 64, 32)
    p = pos.to(DEV)
    one = x.to(DEV).contiguous().requires_grad_()
    y = rotary.rotate(one.expand(30, 5, 64), p, rot)
    assert torch.equal(y.detach().cpu(), ref.rounded(x.expand(30, 5, 64), turn, False))
    g = torch.randn(30, 5, 64, device=DEV)
    y.backward(g)
    want = rotary.rotate(g, p, rot, transpose=True)
    # five terms in fp32, in whatever order: four roundings of partial sums
    assert ((one.grad - want.sum(1, keepdim=True)).abs() <= want.abs().sum(1, keepdim=True) * 8 * 2.0 ** -24).all()
    a = torch.randn(30, 5, 64, device=DEV, requires_grad=True)
    b = a * 2
    z = (b * b).sum()  # saves b
    with torch.no_grad():
        rotary.rotate(b, p, rot, out=b)
    with pytest.raises(RuntimeError):
        z.backward()
