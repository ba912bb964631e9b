"""Rotation and append at the sizes of rotary_cases.py on the GPU, bit for bit against the formula on the CPU."""
import numpy as np
import pytest
import torch

import kvcache_ref
import rotary_ref as ref
from rotary_cases import APPENDS, BF16, TURNS
from scale_search_weights_amd import kvcache, nvfp4, rotary
from test_gpu_rotary import DEV, case, strided

pytestmark = pytest.mark.gpu


def _normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32))


def _turn(rng, c):
    w = torch.from_numpy(1e4 ** (-np.arange(c.pairs) / c.pairs))
    axis = torch.from_numpy(rng.integers(0, c.axes, c.pairs).astype(np.int32)) if c.axes > 1 else None
    pos = torch.from_numpy(rng.integers(-20000, 200000, (c.axes, c.tokens)))
    rot = rotary.Rotary(w.to(DEV), None if axis is None else axis.to(DEV), axes=c.axes, adjacent=c.adjacent,
                        factor=c.factor)
    return rot, pos, ref.turns(pos, w, axis, c.axes)


def _sure(turn, factor):
    """The tokens whose cosines and sines round to fp32 the same way from either side's 64 bits: the kernel's
    angle is good to 2^-50 and its sums to 1e-15 and some roundings of 2^-53, the reference's turn to three
    roundings of 2^-53; together less than 2^-48, times the factor."""
    v, e = torch.view_as_real(turn) * factor, abs(factor) * 2.0 ** -48
    return ((v - e).float() == (v + e).float()).all(-1).all(-1)


def _check(got, x, turn, c, transpose=False):
    """Bit for bit; of a token next to a rounding boundary within the bounds of rotary_ref.rotate."""
    got, sure = got.cpu(), _sure(turn, c.factor)
    assert torch.equal(got[sure], ref.rounded(x, turn, c.adjacent, c.factor, transpose).to(x.dtype)[sure])
    if not sure.all():
        ref.within(got[~sure], *ref.rotate(x[~sure], turn[~sure], c.adjacent, c.factor, transpose))
    assert sure.float().mean() > 0.99


@pytest.mark.parametrize("c", TURNS, ids=[f"{i}" for i in range(len(TURNS))])
def test_rotate(c):
    case(f"rotate {c}")
    rng = np.random.default_rng(c.tokens + c.hd)
    rot, pos, turn = _turn(rng, c)
    x = _normal(rng, c.tokens, c.heads, c.hd).to(torch.bfloat16 if c.dtype == BF16 else torch.float32)
    leaf = strided(x).requires_grad_()
    y = rotary.rotate(leaf, pos.to(DEV), rot)
    _check(y.detach(), x, turn, c)
    g = torch.flip(x, (0,))
    dx, = torch.autograd.grad(y, leaf, strided(g))
    _check(dx, g, turn, c, transpose=True)


@pytest.mark.parametrize("c", APPENDS, ids=[f"{i}" for i in range(len(APPENDS))])
def test_append(c):
    case(f"kv append {c}")
    rng = np.random.default_rng(c.tokens + c.hd)
    dtype = torch.bfloat16 if c.dtype == BF16 else torch.float32
    rot, pos, turn = _turn(rng, c)
    # every head of another size, so that a scale or a row of another head shows
    size = torch.linspace(0.5, 2.0, c.kv_heads).view(1, -1, 1)
    k, v = ((_normal(rng, c.tokens, c.kv_heads, c.hd) * s).to(dtype) for s in (size, size.flip(1)))
    q = _normal(rng, c.tokens, c.heads, c.hd).to(dtype)
    pages = -(-c.tokens // c.page) + 1
    slots = torch.from_numpy(rng.permutation(pages * c.page)[:c.tokens].astype(np.int64))
    slots[torch.from_numpy(rng.random(c.tokens) < 0.1)] = -1
    slots[~_sure(turn, c.factor)] = -1  # a byte next to a boundary could be either
    S_k, S_v = ((x.float().abs().amax((0, 2)) / 2688) for x in (k, v))
    before = [kvcache_ref.any_bytes(rng, (pages, c.kv_heads, c.page, n)) for n in (c.hd // 2, c.hd // 16) * 2]
    cache = kvcache.KVCache(*(t.to(DEV) for t in before), S_k.to(DEV), S_v.to(DEV))
    got = kvcache.append(cache, strided(k), strided(v), slots.to(DEV), pos.to(DEV), rot,
                         q=strided(q) if c.heads else None)
    keep = (slots >= 0).nonzero().squeeze(1)
    page, at = slots[keep] // c.page, slots[keep] % c.page
    for n, x, S in ((0, ref.rounded(k, turn, c.adjacent, c.factor), S_k), (2, v, S_v)):
        for h in range(c.kv_heads):
            codes, scales = nvfp4.quantize(x[:, h].contiguous().to(DEV), S[h:h + 1].to(DEV))
            before[n][page, h, at] = codes.cpu()[keep]
            before[n + 1][page, h, at] = scales.cpu()[keep]
    for name, a, b in zip(("k codes", "k scales", "v codes", "v scales"),
                          (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), before):
        assert torch.equal(a.cpu(), b), name
    if c.heads:
        _check(got, q, turn, c)
    else:
        assert got is None
