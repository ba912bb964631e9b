"""Host side of the key/value cache: exported symbols, and every refusal of the C ABI and of the
Python binding, before anything is launched (no GPU needed)."""
import ctypes
import re

import pytest
import torch

from scale_search_weights_amd import kvcache, nvfp4
from test_abi import EALIGN, EARG, EDTYPE, ENULL, ESHAPE, EWS, FAKE, OK, P, G, _OnGpu1, no_launch  # noqa: F401


@pytest.fixture(scope="module")
def L():
    return kvcache.lib()


def C(codes=FAKE, scales=FAKE, S=FAKE, pages=8, page_size=16, kv_heads=2, head_dim=64, **kw):
    c = kvcache._Cache(codes, scales, codes, scales, S, S, pages, page_size, kv_heads, head_dim)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_exports_what_the_header_declares(L):
    txt = open(nvfp4.HEADER.replace("nvfp4.h", "nvfp4_kv.h")).read()
    names = sorted(set(re.findall(r"NVFP4_API\s+[\w\s\*]*?\b(nvfp4_\w+)\s*\(", txt)))
    assert names == sorted(kvcache._SIGS) and all(hasattr(L, n) for n in names)


BAD_CACHES = [
    (dict(page_size=24), ESHAPE), (dict(page_size=8), ESHAPE), (dict(page_size=1 << 16), ESHAPE),
    (dict(page_size=0), ESHAPE), (dict(head_dim=0), ESHAPE), (dict(head_dim=24), ESHAPE),
    (dict(head_dim=1040), ESHAPE), (dict(pages=-1), ESHAPE), (dict(pages=1 << 31), ESHAPE),
    (dict(kv_heads=-2), ESHAPE), (dict(kv_heads=1 << 16), ESHAPE), (dict(codes=None), ENULL),
    (dict(v_scales=None), ENULL), (dict(S=None), ENULL), (dict(k_codes=FAKE + 8), EALIGN),
    (dict(v_scales=FAKE + 4), EALIGN), (dict(S_k=FAKE + 2), EALIGN)]


@pytest.mark.parametrize("bad,rc", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_every_entry_point_checks_the_cache(L, bad, rc):
    assert L.nvfp4_kv_write(C(**bad), P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE), None) == rc
    assert L.nvfp4_kv_read(C(**bad), P(FAKE), 4, P(FAKE), P(FAKE), 1, None) == rc
    assert attention(L, C(**bad)) == rc
    assert L.nvfp4_kv_attention_workspace_size(C(**bad), 1, 2, 4, 2, 1, 4096, 0) == 0
    assert L.nvfp4_kv_write(None, P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE), None) == ENULL


def test_write_checks(L):
    f = L.nvfp4_kv_write
    assert f(C(), P(FAKE), P(FAKE), 2, 4, 128, 64, 128, 64, P(FAKE), None) == EDTYPE
    assert f(C(), P(FAKE), P(FAKE), 1, -1, 128, 64, 128, 64, P(FAKE), None) == ESHAPE
    assert f(C(), P(FAKE), P(FAKE), 1, 1 << 31, 128, 64, 128, 64, P(FAKE), None) == ESHAPE
    assert f(C(), None, P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE), None) == ENULL
    assert f(C(), P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, None, None) == ENULL
    assert f(C(), P(FAKE), P(FAKE + 8), 1, 4, 128, 64, 128, 64, P(FAKE), None) == EALIGN
    assert f(C(), P(FAKE), P(FAKE), 1, 4, 132, 64, 128, 64, P(FAKE), None) == EALIGN   # bf16: rows of 8
    assert f(C(), P(FAKE), P(FAKE), 0, 4, 128, 64, 128, 66, P(FAKE), None) == EALIGN   # fp32: rows of 4
    assert f(C(), P(FAKE), P(FAKE), 1, 4, -128, 64, 128, 64, P(FAKE), None) == ESHAPE
    assert f(C(), P(FAKE), P(FAKE), 1, 4, 1 << 62, 64, 128, 64, P(FAKE), None) == ESHAPE
    assert f(C(), P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE + 4), None) == EALIGN
    # nothing to do
    assert f(C(), None, None, 1, 0, 128, 64, 128, 64, None, None) == OK
    assert f(C(pages=0, codes=None, scales=None, S=None), P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE), None) == OK
    assert f(C(kv_heads=0), P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE), None) == OK


def test_read_checks(L):
    f = L.nvfp4_kv_read
    assert f(C(), P(FAKE), 4, P(FAKE), P(FAKE), 5, None) == EDTYPE
    assert f(C(), P(FAKE), -4, P(FAKE), P(FAKE), 1, None) == ESHAPE
    assert f(C(), None, 4, P(FAKE), P(FAKE), 1, None) == ENULL
    assert f(C(), P(FAKE), 4, None, None, 1, None) == ENULL
    assert f(C(), P(FAKE), 4, P(FAKE + 8), P(FAKE), 1, None) == EALIGN
    assert f(C(), P(FAKE + 1), 4, P(FAKE), P(FAKE), 1, None) == EALIGN
    assert f(C(), None, 0, None, None, 1, None) == OK


def attention(L, cache, q=FAKE, dtype=1, tokens=2, heads=4, ts=256, hs=64, batch=2, offs=None, max_q=1,
              table=FAKE, width=256, lens=FAKE, max_kv=4096, pp=None, prefix=0, scale=0.1, causal=1,
              out=FAKE, lse=None, ws=FAKE, wsb=1 << 40):
    return L.nvfp4_kv_attention(cache, q, dtype, tokens, heads, ts, hs, batch, offs, max_q, table, width,
                                lens, max_kv, pp, prefix, scale, causal, out, lse, ws, wsb, None)


def test_attention_checks(L):
    for kw, rc in ((dict(dtype=3), EDTYPE), (dict(tokens=-1), ESHAPE), (dict(heads=3), ESHAPE),
                   (dict(heads=-2), ESHAPE), (dict(batch=-1), ESHAPE), (dict(batch=1 << 17), ESHAPE),
                   (dict(max_q=3), ESHAPE), (dict(tokens=3, max_q=1), ESHAPE),
                   (dict(tokens=1 << 30, batch=1, max_q=1 << 30), ESHAPE),
                   (dict(width=-1), ESHAPE), (dict(width=255), ESHAPE), (dict(max_kv=-1), ESHAPE),
                   (dict(max_kv=1 << 31, width=1 << 30), ESHAPE), (dict(prefix=-1), ESHAPE),
                   (dict(prefix=1 << 31), ESHAPE), (dict(scale=float("nan")), EARG),
                   (dict(scale=float("inf")), EARG), (dict(q=None), ENULL), (dict(out=None), ENULL),
                   (dict(table=None), ENULL), (dict(lens=None), ENULL), (dict(prefix=5), ENULL),
                   (dict(q=FAKE + 8), EALIGN), (dict(ts=260), EALIGN), (dict(hs=4), EALIGN),
                   (dict(dtype=0, hs=66), EALIGN), (dict(out=FAKE + 2), EALIGN), (dict(lse=FAKE + 2), EALIGN),
                   (dict(lens=FAKE + 1), EALIGN), (dict(table=FAKE + 2), EALIGN), (dict(offs=FAKE + 2), EALIGN),
                   (dict(pp=FAKE + 2, prefix=4), EALIGN), (dict(ws=None), EWS), (dict(wsb=16), EWS),
                   (dict(ws=FAKE + 8), EALIGN)):
        assert attention(L, C(), **kw) == rc, kw
    assert attention(L, C(head_dim=272, page_size=16)) == ESHAPE  # attention: up to 256
    # nothing to do
    for kw in (dict(tokens=0, max_q=0), dict(heads=0), dict(batch=0, offs=FAKE, tokens=4, max_q=4)):
        assert attention(L, C(), **kw) == OK, kw


def test_attention_workspace(L):
    f = L.nvfp4_kv_attention_workspace_size
    one = f(C(), 1, 1, 4, 1, 1, 100, 0)
    assert one == 0                              # one piece: written at once
    split = f(C(), 1, 1, 4, 1, 1, 100000, 0)
    assert split > 0 and f(C(), 1, 1, 4, 1, 1, 100000, 1000) > split
    assert f(C(), 1, 1, 3, 1, 1, 100, 0) == 0    # what the call refuses


def _bad_calls():
    u8, f32, i32, i64, bf = torch.uint8, torch.float32, torch.int32, torch.int64, torch.bfloat16

    def codes(heads=2, size=16, half=32, dtype=u8):
        return G(4, heads, size, half, dtype=dtype)

    def cache(**kw):
        t = dict(k_codes=codes(), k_scales=codes(half=4), v_codes=codes(), v_scales=codes(half=4), S_k=G(2), S_v=G(2))
        t.update(kw)
        return kvcache.KVCache(*t.values())
    k = G(5, 2, 64)
    q = G(2, 4, 64)
    t, n = G(2, 4, dtype=i32), G(2, dtype=i32)
    att = kvcache.attention
    return [
        ("codes on the host", lambda: cache(k_codes=torch.zeros(4, 2, 16, 32, dtype=u8)), ValueError),
        ("codes int8", lambda: cache(k_codes=codes(dtype=torch.int8)), ValueError),
        ("page size 24", lambda: cache(k_codes=codes(size=24)), ValueError),
        ("head_dim 24", lambda: cache(k_codes=codes(half=12)), ValueError),
        ("scales of another shape", lambda: cache(k_scales=codes(half=8)), ValueError),
        ("value codes of another page count", lambda: cache(v_codes=G(3, 2, 16, 32, dtype=u8)), ValueError),
        ("S_k of one head", lambda: cache(S_k=G(1)), ValueError),
        ("S_v fp64", lambda: cache(S_v=G(2, dtype=torch.float64)), TypeError),
        ("codes not contiguous", lambda: cache(v_codes=G(4, 2, 32, 16, dtype=u8).transpose(2, 3)), ValueError),
        ("k fp16", lambda: kvcache.write(cache(), k.half(), k, G(5, dtype=i64)), TypeError),
        ("v of another dtype", lambda: kvcache.write(cache(), k, k.to(bf), G(5, dtype=i64)), TypeError),
        ("v of fewer tokens", lambda: kvcache.write(cache(), k, k[:4], G(5, dtype=i64)), ValueError),
        ("k of other heads", lambda: kvcache.write(cache(), G(5, 3, 64), k, G(5, dtype=i64)), ValueError),
        ("k of another GPU", lambda: kvcache.write(cache(), G(5, 2, 64, cls=_OnGpu1), k, G(5, dtype=i64)), ValueError),
        ("k strided along head_dim", lambda: kvcache.write(cache(), G(5, 2, 128)[:, :, ::2], k, G(5, dtype=i64)), ValueError),
        ("k rows off 16 bytes", lambda: kvcache.write(cache(), G(5, 2, 65)[:, :, :64], k, G(5, dtype=i64)), ValueError),
        ("slots int32", lambda: kvcache.write(cache(), k, k, G(5, dtype=i32)), TypeError),
        ("slots too few", lambda: kvcache.write(cache(), k, k, G(4, dtype=i64)), ValueError),
        ("read slots on the host", lambda: kvcache.read(cache(), torch.zeros(3, dtype=i64)), ValueError),
        ("read to fp16", lambda: kvcache.read(cache(), G(3, dtype=i64), torch.float16), TypeError),
        ("q of another head_dim", lambda: att(cache(), G(2, 4, 32), t, n), ValueError),
        ("3 heads over 2", lambda: att(cache(), G(2, 3, 64), t, n), ValueError),
        ("q on the host", lambda: att(cache(), torch.zeros(2, 4, 64), t, n), ValueError),
        ("q rows off 16 bytes", lambda: att(cache(), G(2, 4, 66)[:, :, 2:], t, n), ValueError),
        ("head_dim over 256", lambda: att(cache(k_codes=codes(half=136), k_scales=codes(half=17), v_codes=codes(half=136),
                                                v_scales=codes(half=17)), G(2, 4, 272), t, n), ValueError),
        ("table without lengths", lambda: att(cache(), q, t), ValueError),
        ("table int64", lambda: att(cache(), q, t.long(), n), TypeError),
        ("table of one dimension", lambda: att(cache(), q, n, n), TypeError),
        ("lengths of three sequences", lambda: att(cache(), q, t, G(3, dtype=i32)), ValueError),
        ("tokens no multiple of the batch", lambda: att(cache(), G(3, 4, 64), t, n), ValueError),
        ("max_q other than tokens / batch", lambda: att(cache(), q, t, n, max_q=2), ValueError),
        ("offsets of three sequences", lambda: att(cache(), q, t, n, q_offsets=G(4, dtype=i32)), ValueError),
        ("negative max_kv", lambda: att(cache(), q, t, n, max_kv=-1), ValueError),
        ("prefix without pages", lambda: att(cache(), q, t, n, prefix_len=3), TypeError),
        ("prefix longer than its pages", lambda: att(cache(), q, t, n, prefix_pages=G(2, dtype=i32), prefix_len=33), ValueError),
        ("out of another dtype", lambda: att(cache(), q, t, n, out=G(2, 4, 64, dtype=bf)), TypeError),
        ("out too small", lambda: att(cache(), q, t, n, out=G(1, 4, 64)), ValueError),
    ]


@pytest.mark.parametrize("what,call,exc", _bad_calls(), ids=[c[0] for c in _bad_calls()])
def test_binding_refuses(no_launch, monkeypatch, what, call, exc):  # noqa: F811
    monkeypatch.setattr(kvcache, "_bound", None)
    with pytest.raises(exc):
        call()
