"""Host side of the rotation, the append and windowed attention: exported symbols, and every refusal of the C
ABI and of the Python binding, before anything is launched (no GPU needed)."""
import ctypes
import re

import pytest
import torch

from scale_search_weights_amd import kvcache, nvfp4, rotary
from test_abi import EALIGN, EARG, EDTYPE, ENULL, ESHAPE, EWS, FAKE, OK, P, G, _OnGpu1, no_launch  # noqa: F401
from test_kvcache_host import BAD_CACHES, C

BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    kvcache.lib()
    return rotary.lib()


def R(inv_freq=FAKE, axis=None, pairs=32, axes=1, adjacent=0, factor=1.0):
    return ctypes.byref(rotary._Rotary(inv_freq, axis, pairs, axes, factor, adjacent))


def test_exports_what_the_header_declares(L):
    txt = open(nvfp4.HEADER.replace("nvfp4.h", "nvfp4_rotary.h")).read()
    names = sorted(set(re.findall(r"NVFP4_API\s+[\w\s\*]*?\b(nvfp4_\w+)\s*\(", txt)))
    assert names == sorted(rotary._SIGS) and all(hasattr(L, n) for n in names)


def rotate(L, r=None, pos=FAKE, ps=0, x=FAKE, dtype=1, tokens=4, heads=2, hd=64, ts=128, hs=64, out=FAKE, ots=128, ohs=64,
           t=0):
    return L.nvfp4_rotate(r or R(), pos, ps, x, dtype, tokens, heads, hd, ts, hs, out, ots, ohs, t, None)


BAD_ROTARY = [(dict(pairs=0), ESHAPE), (dict(pairs=-4), ESHAPE), (dict(pairs=516), ESHAPE), (dict(pairs=36), ESHAPE),
              (dict(axes=0), ESHAPE), (dict(axes=17), ESHAPE), (dict(factor=float("nan")), EARG),
              (dict(factor=float("inf")), EARG), (dict(inv_freq=None), ENULL), (dict(inv_freq=FAKE + 4), EALIGN),
              (dict(axis=FAKE + 2), EALIGN)]


@pytest.mark.parametrize("bad,rc", BAD_ROTARY, ids=[str(b[0]) for b in BAD_ROTARY])
def test_both_check_the_rotary(L, bad, rc):
    assert rotate(L, R(**bad)) == rc
    assert append(L, r=R(**bad)) == rc


def test_rotate_checks(L):
    for kw, rc in ((dict(dtype=2), EDTYPE), (dict(hd=0), ESHAPE), (dict(hd=60), ESHAPE), (dict(hd=56), ESHAPE),
                   (dict(hd=1032), ESHAPE), (dict(tokens=-1), ESHAPE), (dict(tokens=1 << 31), ESHAPE),
                   (dict(heads=-1), ESHAPE), (dict(heads=1 << 16), ESHAPE), (dict(x=None), ENULL), (dict(out=None), ENULL),
                   (dict(pos=None), ENULL), (dict(pos=FAKE + 4), EALIGN), (dict(ps=-1), ESHAPE), (dict(ps=BIG), ESHAPE),
                   (dict(x=FAKE + 8), EALIGN), (dict(out=FAKE + 8), EALIGN), (dict(ts=132), EALIGN), (dict(hs=68), EALIGN),
                   (dict(dtype=0, ts=130), EALIGN), (dict(ts=-128), ESHAPE), (dict(ts=BIG), ESHAPE), (dict(ots=BIG), ESHAPE),
                   # rows of the output on top of each other
                   (dict(ots=0), ESHAPE), (dict(ohs=0), ESHAPE), (dict(ots=64), ESHAPE), (dict(ots=56, ohs=512), ESHAPE),
                   (dict(ots=64, ohs=192), ESHAPE), (dict(ots=96), ESHAPE)):
        assert rotate(L, **kw) == rc, kw
    assert L.nvfp4_rotate(None, FAKE, 0, FAKE, 1, 4, 2, 64, 128, 64, FAKE, 128, 64, 0, None) == ENULL
    # nothing to do
    for kw in (dict(tokens=0, x=None, out=None, pos=None), dict(heads=0, x=None, out=None)):
        assert rotate(L, **kw) == OK, kw


def append(L, c=None, r=None, pos=FAKE, ps=0, q=FAKE, k=FAKE, v=FAKE, dtype=1, tokens=4, heads=4, qs=(256, 64), ks=(128, 64),
           vs=(128, 64), out=FAKE, os=(256, 64), slots=FAKE):
    return L.nvfp4_kv_append(c or C(), r or R(), pos, ps, q, k, v, dtype, tokens, heads, *qs, *ks, *vs, out, *os, slots, None)


@pytest.mark.parametrize("bad,rc", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_append_and_window_check_the_cache(L, bad, rc):
    assert append(L, C(**bad)) == rc
    assert window(L, C(**bad)) == rc
    assert L.nvfp4_kv_window_attention_workspace_size(C(**bad), 1, 2, 4, 2, 1, 40960, 8192, 4) == 0


def test_append_checks(L):
    for kw, rc in ((dict(dtype=7), EDTYPE), (dict(tokens=-1), ESHAPE), (dict(tokens=1 << 31), ESHAPE), (dict(heads=-1), ESHAPE),
                   (dict(heads=1 << 16), ESHAPE), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(slots=None), ENULL),
                   (dict(q=None), ENULL), (dict(out=None), ENULL), (dict(pos=None), ENULL), (dict(pos=FAKE + 1), EALIGN),
                   (dict(ps=-8), ESHAPE), (dict(slots=FAKE + 4), EALIGN), (dict(q=FAKE + 8), EALIGN), (dict(k=FAKE + 8), EALIGN),
                   (dict(v=FAKE + 8), EALIGN), (dict(out=FAKE + 8), EALIGN), (dict(qs=(260, 64)), EALIGN),
                   (dict(ks=(128, 4)), EALIGN), (dict(vs=(-128, 64)), ESHAPE), (dict(vs=(BIG, 64)), ESHAPE),
                   (dict(os=(256, 0)), ESHAPE), (dict(os=(64, 64)), ESHAPE), (dict(os=(256, 32)), ESHAPE)):
        assert append(L, **kw) == rc, kw
    assert append(L, r=R(pairs=12)) == ESHAPE   # pairs in multiples of 8 here
    assert rotate(L, R(pairs=12), tokens=0) == OK
    assert L.nvfp4_kv_append(C(), None, FAKE, 0, None, FAKE, FAKE, 1, 4, 0, 0, 0, 128, 64, 128, 64, None, 0, 0, FAKE, None) == ENULL
    # nothing to do
    assert append(L, tokens=0, q=None, k=None, v=None, slots=None, out=None, pos=None) == OK
    none = C(pages=0, codes=None, scales=None, S=None)
    assert append(L, none, heads=0, q=None, out=None, k=None, v=None, slots=None) == OK
    assert append(L, C(kv_heads=0), heads=0, q=None, out=None) == OK


def window(L, cache=None, q=FAKE, dtype=1, tokens=2, heads=4, ts=256, hs=64, batch=2, offs=None, max_q=1, table=FAKE, width=2560,
           lens=FAKE, max_kv=40960, w=8192, sinks=4, scale=0.1, out=FAKE, lse=None, ws=FAKE, wsb=1 << 40):
    return L.nvfp4_kv_window_attention(cache or C(), q, dtype, tokens, heads, ts, hs, batch, offs, max_q, table, width, lens, max_kv,
                                       w, sinks, scale, out, lse, ws, wsb, None)


def test_window_checks(L):
    for kw, rc in ((dict(dtype=3), EDTYPE), (dict(tokens=-1), ESHAPE), (dict(heads=3), ESHAPE), (dict(batch=1 << 17), ESHAPE),
                   (dict(max_q=3), ESHAPE), (dict(tokens=3, max_q=1), ESHAPE), (dict(width=-1), ESHAPE), (dict(width=2559), ESHAPE),
                   (dict(max_kv=-1), ESHAPE), (dict(max_kv=1 << 31, width=1 << 30), ESHAPE), (dict(w=0), ESHAPE),
                   (dict(w=-1), ESHAPE), (dict(w=(1 << 30) + 1), ESHAPE), (dict(sinks=-1), ESHAPE),
                   (dict(sinks=(1 << 30) + 1), ESHAPE), (dict(scale=float("nan")), EARG), (dict(q=None), ENULL),
                   (dict(out=None), ENULL), (dict(table=None), ENULL), (dict(lens=None), ENULL), (dict(q=FAKE + 8), EALIGN),
                   (dict(ts=260), EALIGN), (dict(out=FAKE + 2), EALIGN), (dict(lse=FAKE + 2), EALIGN),
                   (dict(lens=FAKE + 1), EALIGN), (dict(table=FAKE + 2), EALIGN), (dict(offs=FAKE + 2), EALIGN),
                   (dict(ws=None), EWS), (dict(wsb=16), EWS), (dict(ws=FAKE + 8), EALIGN)):
        assert window(L, **kw) == rc, kw
    assert window(L, C(head_dim=272)) == ESHAPE
    for kw in (dict(tokens=0, max_q=0), dict(heads=0), dict(batch=0, offs=FAKE, tokens=4, max_q=4)):
        assert window(L, **kw) == OK, kw


def test_window_workspace(L):
    f = L.nvfp4_kv_window_attention_workspace_size
    assert f(C(), 1, 1, 4, 1, 1, 100000, 64, 4) == 0               # one piece
    need = f(C(), 1, 1, 4, 1, 1, 100000, 8192, 4)
    assert need > 0 and f(C(), 1, 1, 4, 1, 1, 1 << 30, 8192, 4) == need   # the context does not count
    for bad in ((1, 1, 3, 1, 1, 100, 64, 4), (1, 1, 4, 1, 1, 100, 0, 4), (1, 1, 4, 1, 1, 100, 64, -1)):
        assert f(C(), *bad) == 0
    assert f(C(), 1, 200, 4, 1, 200, 0, 64, 4) == 0                # no tokens are cached


def _bad_calls():
    f32, i32, i64, f64, bf = torch.float32, torch.int32, torch.int64, torch.float64, torch.bfloat16
    u8 = torch.uint8

    def rot(pairs=32, axis=None, **kw):
        return rotary.Rotary(G(pairs, dtype=f64), axis, **kw)

    def cache():
        return kvcache.KVCache(G(4, 2, 16, 32, dtype=u8), G(4, 2, 16, 4, dtype=u8), G(4, 2, 16, 32, dtype=u8),
                               G(4, 2, 16, 4, dtype=u8), G(2), G(2))
    x, p, s = G(5, 2, 64), G(5, dtype=i64), G(5, dtype=i64)
    turn, app = rotary.rotate, kvcache.append
    q, t, n = G(2, 4, 64), G(2, 4, dtype=i32), G(2, dtype=i32)
    att = kvcache.attention
    return [
        ("frequencies fp32", lambda: rotary.Rotary(G(32)), TypeError),
        ("frequencies on the host", lambda: rotary.Rotary(torch.zeros(32, dtype=f64)), ValueError),
        ("frequencies of two dimensions", lambda: rotary.Rotary(G(4, 8, dtype=f64)), TypeError),
        ("frequencies to be trained", lambda: rotary.Rotary(G(32, dtype=f64).requires_grad_()), ValueError),
        ("30 pairs", lambda: rot(30), ValueError),
        ("516 pairs", lambda: rot(516), ValueError),
        ("axis of other length", lambda: rot(32, G(31, dtype=i32)), TypeError),
        ("axis int64", lambda: rot(32, G(32, dtype=i64)), TypeError),
        ("axis of another GPU", lambda: rot(32, G(32, dtype=i32, cls=_OnGpu1)), ValueError),
        ("axes without axis", lambda: rot(32, axes=3), ValueError),
        ("no axes", lambda: rot(32, G(32, dtype=i32), axes=0), ValueError),
        ("17 axes", lambda: rot(32, G(32, dtype=i32), axes=17), ValueError),
        ("factor NaN", lambda: rot(32, factor=float("nan")), ValueError),
        ("rotary_dim 60", lambda: rotary.Rotary.create(60), ValueError),
        ("sections of 60 pairs", lambda: rotary.Rotary.create(128, sections=(16, 24, 20)), ValueError),
        ("no sections", lambda: rotary.Rotary.create(128, sections=()), ValueError),
        ("no rotary", lambda: turn(x, p, None), TypeError),
        ("append without rotary", lambda: app(cache(), x, x, s, p, None), TypeError),
        ("x fp16", lambda: turn(x.half(), p, rot()), TypeError),
        ("x on the host", lambda: turn(torch.zeros(5, 2, 64), p, rot()), ValueError),
        ("x of two dimensions", lambda: turn(G(5, 64), p, rot()), ValueError),
        ("x narrower than the pairs", lambda: turn(G(5, 2, 56), p, rot()), ValueError),
        ("x of 1032 channels", lambda: turn(G(5, 2, 1032), p, rot()), ValueError),
        ("x strided along head_dim", lambda: turn(G(5, 2, 128)[:, :, ::2], p, rot()), ValueError),
        ("x rows off 16 bytes", lambda: turn(G(5, 2, 65)[:, :, :64], p, rot()), ValueError),
        ("positions int32", lambda: turn(x, G(5, dtype=i32), rot()), TypeError),
        ("positions of four tokens", lambda: turn(x, G(4, dtype=i64), rot()), ValueError),
        ("positions of two axes", lambda: turn(x, G(2, 5, dtype=i64), rot()), ValueError),
        ("positions of one axis for two", lambda: turn(x, p, rot(32, G(32, dtype=i32), axes=2)), ValueError),
        ("positions strided", lambda: turn(x, G(10, dtype=i64)[::2], rot()), ValueError),
        ("positions on the host", lambda: turn(x, torch.zeros(5, dtype=i64), rot()), ValueError),
        ("positions of another GPU", lambda: turn(x, G(5, dtype=i64, cls=_OnGpu1), rot()), ValueError),
        ("out of another type", lambda: turn(x, p, rot(), out=G(5, 2, 64, dtype=bf)), ValueError),
        ("out of another shape", lambda: turn(x, p, rot(), out=G(5, 2, 72)), ValueError),
        ("out for gradients", lambda: turn(G(5, 2, 64).requires_grad_(), p, rot(), out=x), ValueError),
        ("append: 36 pairs of 64", lambda: app(cache(), x, x, s, p, rot(36)), ValueError),
        ("append: 28 pairs", lambda: app(cache(), x, x, s, p, rot(28)), ValueError),
        ("append: v of another type", lambda: app(cache(), x, x.to(bf), s, p, rot()), TypeError),
        ("append: slots int32", lambda: app(cache(), x, x, G(5, dtype=i32), p, rot()), TypeError),
        ("append: slots too few", lambda: app(cache(), x, x, G(4, dtype=i64), p, rot()), ValueError),
        ("append: positions too few", lambda: app(cache(), x, x, s, G(4, dtype=i64), rot()), ValueError),
        ("append: q of another type", lambda: app(cache(), x, x, s, p, rot(), q=G(5, 4, 64, dtype=bf)), TypeError),
        ("append: q of four tokens", lambda: app(cache(), x, x, s, p, rot(), q=G(4, 4, 64)), ValueError),
        ("append: q of another head_dim", lambda: app(cache(), x, x, s, p, rot(), q=G(5, 4, 32)), ValueError),
        ("append: q_out of another shape", lambda: app(cache(), x, x, s, p, rot(), q=G(5, 4, 64), q_out=x), ValueError),
        ("append: q_out without q", lambda: app(cache(), x, x, s, p, rot(), q_out=x), ValueError),
        ("append: k of other heads", lambda: app(cache(), G(5, 3, 64), x, s, p, rot()), ValueError),
        ("window 0", lambda: att(cache(), q, t, n, window=0), ValueError),
        ("window past 2^30", lambda: att(cache(), q, t, n, window=1 << 31), ValueError),
        ("sinks -1", lambda: att(cache(), q, t, n, window=4, sinks=-1), ValueError),
        ("sinks without a window", lambda: att(cache(), q, t, n, sinks=4), ValueError),
        ("window not causal", lambda: att(cache(), q, t, n, window=4, causal=False), ValueError),
        ("window and prefix", lambda: att(cache(), q, t, n, window=4, prefix_pages=G(1, dtype=i32), prefix_len=3), ValueError),
        ("window of half a token", lambda: att(cache(), q, t, n, window=4.5), TypeError),
    ]


@pytest.mark.parametrize("what,call,exc", _bad_calls(), ids=[c[0] for c in _bad_calls()])
def test_binding_refuses(no_launch, monkeypatch, what, call, exc):  # noqa: F811
    monkeypatch.setattr(kvcache, "_bound", None)
    monkeypatch.setattr(rotary, "_bound", None)
    with pytest.raises(exc):
        call()
