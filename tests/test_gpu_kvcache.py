"""The NVFP4 key/value cache on the GPU against 64-bit references on the CPU.

write and read are exact: codes, block bytes and dequantised values have to agree bit for bit
with the quantiser's definition. attention's bounds, per output element:
  * a probability is rounded to fp16 (relative 2^-11) for bf16 queries, to 22 bits for fp32;
  * a score's error is at most 2^-19 B, B = max_t |scale| sum_d |q_d k_td|: fp32 sums of at most
    32 partial sums of 16 products (2^-24 each, twice), the 22-bit queries (2^-22), and the
    fp32 factor scale S log2(e) and exp2 (a few 2^-23);
  * the sum over tokens is fp32 (within 2^-20 of A for the lengths here, A = sum_t p_t |v_t|);
  * the output is rounded to its type.
An error d of a score changes p by a factor e^d, in the numerator and in the denominator:
  |out - ref| <= A (2 (2^-19 B) 1.05 + 2^-11 or 2^-21, + 2^-20) + |ref| 2^-8 (bf16) or 2^-22 (fp32)
where the bf16 output's half ulp 2^-9 is doubled for values next to a rounding boundary.
This leaves out fp16's smallest step, which matters only where a few tokens hold nearly the whole
row and are zero in a channel. The probabilities are held so that the largest is at least 2^7
(2^13 for fp32), and half of the smallest step is 2^-25, so each may be off by 2^-32 (2^-38) of
the largest: with floor=True, 2^-32 or 2^-38 times V = sum_t |v_t| is added.
"""
import math

import numpy as np
import pytest
import torch

import kvcache_ref as ref
from scale_search_weights_amd import kvcache, nvfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def case(msg):
    print(f"[case] {msg}", flush=True)


def on_gpu(c):
    kc, ks, vc, vs, S_k, S_v, _ = c["cache"]
    return kvcache.KVCache(*(t.to(DEV) for t in (kc, ks, vc, vs, S_k, S_v)))


def strided(q):
    """q on the GPU with the strides it has here."""
    if q.numel() == 0:
        return q.to(DEV)
    base = torch.empty(q.stride(0) * q.shape[0], dtype=q.dtype, device=DEV)
    y = base.as_strided(q.shape, q.stride())
    y.copy_(q)
    return y


def attend(c, cache=None, causal=True, scale=None, **kw):
    q = strided(c["q"])
    own = c["max_kv"] > 0
    return kvcache.attention(
        cache or on_gpu(c), q, c["table"].to(DEV) if own else None,
        c["kv_lens"].to(DEV) if own else None, q_offsets=c["q_offsets"].to(DEV), max_q=c["max_q"],
        max_kv=c["max_kv"] if own else None,
        prefix_pages=c["prefix_pages"].to(DEV) if c["prefix_len"] else None,
        prefix_len=c["prefix_len"], causal=causal, scale=scale, return_lse=True, **kw)


def check(c, got, causal=True, scale=None, floor=False):
    out, lse = (t.cpu() for t in got)
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    o, z, A, B, V = ref.attention(c["cache"], c["q"], c["table"], c["kv_lens"] if c["max_kv"] else None,
                               c["q_offsets"], c["prefix_pages"], c["prefix_len"], scale, causal)
    bf = out.dtype == BF
    d = 2 * 1.05 * 2.0 ** -19 * B.unsqueeze(-1) + (2.0 ** -11 if bf else 2.0 ** -21) + 2.0 ** -20
    tol = A * d + o.abs() * (2.0 ** -8 if bf else 2.0 ** -22)
    if floor:
        tol += V * (2.0 ** -32 if bf else 2.0 ** -38)
    err = (out.double() - o).abs()
    assert torch.isfinite(out.float()).all()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0, (worst, err.max().item(), tol[err > tol][:3])
    empty = torch.isneginf(z)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    dl = ((lse.double() - z).abs() - (2.0 ** -19 * B + 2.0 ** -19 + 2.0 ** -22 * z.abs()))[~empty]
    assert not dl.numel() or dl.max() <= 0, dl.max()
    return o


# ------------------------------------------------------------------------------ write, read

def _kv(seed, dtype, tokens, heads, hd, ties=False):
    rng = np.random.default_rng(seed)
    if ties:  # multiples of a quarter grid step at S = 2^-k: many exact midpoints
        x = rng.integers(-3000, 3001, (tokens, 2 * heads + 1, hd)).astype(np.float32) / 128
        x *= np.exp2(rng.integers(-9, 2, (tokens, 2 * heads + 1, 1))).astype(np.float32)
    else:
        x = rng.standard_normal((tokens, 2 * heads + 1, hd)).astype(np.float32)
        x[:, :, rng.integers(0, hd, 2)] *= 30
    x[rng.random(x.shape[:2]) < 0.05] = 0.0
    x[0, 0, :16] = -0.0
    x = torch.from_numpy(x).to(dtype)
    return x[:, :heads], x[:, heads:2 * heads]


@pytest.mark.parametrize("dtype,tokens,heads,hd,page_size,S,ties", [
    (BF, 1, 1, 16, 16, None, False), (BF, 33, 8, 128, 16, None, False), (F32, 100, 5, 80, 32, None, False),
    (BF, 257, 3, 64, 64, 1 / 512, True), (F32, 130, 2, 256, 16, 0.75 / 256, True), (BF, 70, 4, 96, 128, 0.0013, True),
    (F32, 19, 1, 1024, 16, None, False), (BF, 21, 2, 1008, 16, None, False), (BF, 5000, 2, 112, 256, None, False)])
def test_write_matches_the_quantiser_and_read_dequantises(dtype, tokens, heads, hd, page_size, S, ties):
    case(f"kv write/read {dtype} {tokens}x{heads}x{hd}, pages of {page_size}")
    k, v = _kv(tokens + hd, dtype, tokens, heads, hd, ties)
    rng = np.random.default_rng(3)
    pages = -(-tokens // page_size) + 1
    slots = torch.from_numpy(rng.permutation(pages * page_size)[:tokens].astype(np.int64))
    skip = torch.from_numpy(rng.random(tokens) < 0.15)
    if tokens > 3:
        slots[1], skip[1] = pages * page_size, True  # one past the end
    slots[skip & (slots < pages * page_size)] = -1
    Sk = torch.full((heads,), S) if S else (k.float().abs().amax((0, 2)) / 2688).clamp(min=1e-6)
    Sv = torch.full((heads,), S) if S else (v.float().abs().amax((0, 2)) / 2688).clamp(min=1e-6)
    before = [ref.any_bytes(rng, (pages, heads, page_size, n)) for n in (hd // 2, hd // 16) * 2]
    cache = kvcache.KVCache(*(t.to(DEV) for t in before), Sk.to(DEV), Sv.to(DEV))
    kvcache.write(cache, strided(k), strided(v), slots.to(DEV))
    got = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    for n, x, sc in ((0, k, Sk), (2, v, Sv)):
        # the library's quantiser, head by head (its own tests hold it to the oracle)
        want_c, want_s = before[n].clone(), before[n + 1].clone()
        keep = (~skip).nonzero().squeeze(1)
        for h in range(heads):
            c, s = nvfp4.quantize(x[:, h].contiguous().to(DEV), sc[h:h + 1].to(DEV))
            want_c[slots[keep] // page_size, h, slots[keep] % page_size] = c.cpu()[keep]
            want_s[slots[keep] // page_size, h, slots[keep] % page_size] = s.cpu()[keep]
        assert torch.equal(got[n], want_c) and torch.equal(got[n + 1], want_s)
    for out in (BF, F32):
        ys = kvcache.read(cache, slots.to(DEV), out)
        for y, n, sc in ((ys[0], 0, Sk), (ys[1], 2, Sv)):
            at = slots.clamp(0, pages * page_size - 1)
            want = ref.values(got[n][at // page_size, :, at % page_size],
                              got[n + 1][at // page_size, :, at % page_size], sc.view(1, -1, 1)).float()
            want[skip] = 0
            assert torch.equal(y.cpu(), want.to(out))


def test_write_decides_exactly(orc):
    """Against the CPU oracle at a head scale with a full 24-bit significand."""
    case("kv write against the oracle")
    k, v = _kv(11, F32, 64, 2, 64, ties=True)
    S = torch.tensor([0.00371234, 0.0123457])
    cache = kvcache.KVCache.empty(4, 16, 2, 64, S.to(DEV), S.to(DEV))
    kvcache.write(cache, strided(k), strided(v), torch.arange(64, device=DEV))
    for h in range(2):
        _, codes, scales = orc.fakequant(k[:, h].contiguous().numpy(), float(S[h]))
        assert np.array_equal(cache.k_codes[:, h].reshape(64, 32).cpu().numpy(), codes)
        assert np.array_equal(cache.k_scales[:, h].reshape(64, 4).cpu().numpy(), scales)


def test_read_of_any_bytes():
    """Sign bits of scale bytes are ignored and 0x7F is zero, as in dequantize."""
    case("kv read of arbitrary cache bytes")
    rng = np.random.default_rng(5)
    t = [ref.any_bytes(rng, (3, 2, 16, n)) for n in (24, 3, 24, 3)]
    S = torch.tensor([0.01, 3.0])
    cache = kvcache.KVCache(*(x.to(DEV) for x in t), S.to(DEV), S.to(DEV))
    slots = torch.arange(48, device=DEV)
    k, v = kvcache.read(cache, slots, F32)
    for y, c, s in ((k, t[0], t[1]), (v, t[2], t[3])):
        want = ref.values(c, s, S.view(1, 2, 1, 1)).float().transpose(1, 2).reshape(48, 2, 48)
        assert torch.equal(y.cpu(), want)


# -------------------------------------------------------------------------------- attention

SHAPES = [
    # dtype, q_lens, kv_lens, heads, kv_heads, hd, page_size, prefix, causal
    (BF, [1], [1], 1, 1, 64, 16, 0, True),
    (BF, [1], [1000], 32, 8, 128, 16, 0, True),
    (BF, [1] * 5, [17, 0, 300, 16, 129], 8, 2, 128, 16, 0, True),
    (BF, [1] * 4, [40, 0, 31, 700], 16, 2, 128, 32, 77, True),
    (BF, [1] * 3, [0, 0, 0], 4, 4, 64, 16, 0, True),
    (BF, [1] * 3, [0, 0, 0], 4, 4, 64, 16, 33, True),
    (BF, [3, 0, 5, 1], [3, 0, 900, 64], 12, 4, 128, 64, 0, True),
    (BF, [4, 2], [2, 300], 4, 1, 96, 16, 0, True),       # more queries than cached tokens
    (BF, [4, 2], [2, 300], 4, 1, 96, 16, 50, True),
    (BF, [7, 9, 40], [100, 9, 333], 28, 4, 128, 16, 0, True),
    (BF, [130], [130], 6, 2, 128, 16, 0, True),
    (BF, [70, 200], [500, 200], 8, 2, 64, 32, 19, True),
    (BF, [33, 65], [150, 90], 10, 5, 80, 16, 100, False),
    (BF, [2, 2], [1500, 37], 20, 20, 64, 16, 0, False),
    (BF, [1] * 40, [100] * 39 + [2], 8, 2, 128, 16, 900, True),
    (BF, [5], [200], 8, 1, 256, 16, 40, True),
    (BF, [100], [260], 4, 2, 256, 128, 0, True),
    (BF, [6], [90], 3, 3, 16, 16, 20, True),
    (BF, [6], [90], 6, 3, 48, 16, 20, True),
    (BF, [37], [90], 4, 2, 160, 16, 20, True),
    (BF, [37], [90], 4, 2, 240, 16, 0, False),
    (F32, [1], [333], 8, 2, 128, 16, 0, True),
    (F32, [4, 1, 3], [400, 0, 77], 8, 1, 256, 16, 65, True),
    (F32, [50, 90], [180, 90], 6, 2, 64, 16, 31, True),
    (F32, [300], [420], 4, 1, 128, 64, 0, True),
    (F32, [20], [80], 5, 5, 112, 16, 0, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_attention(shape):
    dtype, q_lens, kv_lens, heads, kv_heads, hd, ps, prefix, causal = shape
    case(f"kv attention {shape}")
    c = ref.make(len(q_lens) * 100 + hd, dtype, q_lens, kv_lens, heads, kv_heads, hd, ps, prefix)
    check(c, attend(c, causal=causal), causal)


def test_attention_long_context_split():
    case("kv attention: 40000 tokens, one query; 3 heads a group")
    c = ref.make(1, BF, [1], [40000], 6, 2, 128, 64)
    check(c, attend(c))


LARGE = [(BF, 40.0, None), (F32, 40.0, None), (BF, 1e30, 1e-30), (BF, 1e-30, 1e30), (F32, 1e-20, 1e20),
         (BF, 1.0, 0.0), (BF, 1.0, -0.2), (F32, 0.0, None)]
VANISH = pytest.mark.xfail(strict=True, reason="probabilities under 2^-32 (fp32: 2^-38) of the row's "
                           "largest vanish in fp16: channels where the largest tokens are zero")


@pytest.mark.parametrize("dtype,qs,scale", [pytest.param(*x, marks=VANISH if x[1] == 40.0 else ()) for x in LARGE])
def test_attention_large_scores_and_scales(dtype, qs, scale):
    """Scores in the hundreds (one token takes the row), tiny and huge queries, scale 0 and < 0."""
    case(f"kv attention, q ~ {qs}, scale {scale}, {dtype}")
    c = ref.make(9, dtype, [2, 1], [210, 64], 8, 2, 128, 16, 40, q_scale=qs)
    check(c, attend(c, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,qs,scale", LARGE)
def test_attention_large_scores_down_to_the_smallest_step(dtype, qs, scale):
    case(f"kv attention, q ~ {qs}, scale {scale}, {dtype}, with fp16's smallest step in the bound")
    c = ref.make(9, dtype, [2, 1], [210, 64], 8, 2, 128, 16, 40, q_scale=qs)
    check(c, attend(c, scale=scale), scale=scale, floor=True)


def test_attention_scores_rise_and_fall():
    """Keys scaled so that the running maximum climbs over the whole sequence, and the reverse."""
    for flip in (False, True):
        case(f"kv attention, {'falling' if flip else 'rising'} scores")
        c = ref.make(21, BF, [1, 3], [900, 700], 4, 2, 64, 16)
        ks = c["cache"][1]
        for b, m in enumerate((900, 700)):
            t = torch.arange(m)
            byte = (0x10 + (t * 0x58) // m).to(torch.uint8)
            byte = byte.flip(0) if flip else byte
            ks[c["table"][b].long()[t // 16], :, t % 16] = byte.view(-1, 1, 1)
        check(c, attend(c))


def test_hidden_pages():
    """Page ids outside the cache hide their tokens; a row may be left with none."""
    case("kv attention with page ids outside the cache")
    c = ref.make(31, BF, [1, 1, 2], [100, 40, 90], 4, 2, 128, 16, 64)
    c["table"][0, 2], c["table"][0, 5] = -1, 10 ** 6
    c["table"][1, :] = -5
    c["prefix_pages"][1] = 1 << 30
    check(c, attend(c))
    c["prefix_len"] = 0
    o = check(c, attend(c))
    assert (o[1] == 0).all()


def test_bytes_beyond_the_length_do_not_matter():
    case("kv attention: bytes of unused slots")
    c = ref.make(41, BF, [1, 5], [37, 130], 8, 2, 128, 64, 21)
    a = attend(c)
    kc, ks, vc, vs, S_k, S_v, ps = c["cache"]
    used = torch.zeros(kc.shape[0], ps, dtype=torch.bool)
    for pages, n in ((c["prefix_pages"], 21), (c["table"][0], 37), (c["table"][1], 130)):
        t = torch.arange(n)
        used[pages.long()[t // ps], t % ps] = True
    for x, fill in ((kc, 0xFF), (vc, 0xF7), (ks, 0x7F), (vs, 0xFF)):
        x.transpose(1, 2)[~used] = fill
    b = attend(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_lengths_on_the_device_may_be_shorter_than_the_bounds():
    """max_q and max_kv are bounds, not lengths; lengths over max_kv are cut."""
    case("kv attention with loose bounds")
    c = ref.make(51, BF, [1, 2, 1], [50, 2, 130], 8, 4, 64, 16, 30)
    want = attend(c)
    loose = dict(c, max_q=4, max_kv=c["table"].shape[1] * 16)
    got = attend(loose)
    assert torch.allclose(want[0].float(), got[0].float(), atol=2.0 ** -7)
    check(c, got)
    cut = dict(c, kv_lens=torch.tensor([50, -7, 1 << 30], dtype=torch.int32))
    got = attend(cut)
    check(dict(c, kv_lens=torch.tensor([50, 0, 130], dtype=torch.int32)), got)


def test_repeatable_on_another_stream_and_in_a_graph():
    case("kv attention: same bits again, on a side stream, in a graph")
    c = ref.make(61, BF, [1] * 6, [700, 3, 0, 250, 64, 900], 8, 2, 128, 16, 333)
    cache, q = on_gpu(c), strided(c["q"])
    table, lens, pp = c["table"].to(DEV), c["kv_lens"].to(DEV), c["prefix_pages"].to(DEV)

    def run(out=None):
        return kvcache.attention(cache, q, table, lens, max_kv=c["max_kv"], prefix_pages=pp, prefix_len=333,
                                 out=out)
    want = run()
    for _ in range(3):
        assert torch.equal(run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for n in range(4):
        q.copy_(torch.randn_like(q.float()).to(BF))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        assert torch.equal(out, eager), n


def test_offsets_beyond_32_bits():
    """A cache of over 2^32 code bytes a tensor, its last pages in use."""
    case("kv cache of more than 4 GiB of codes")
    heads, hd, ps = 2, 256, 512
    pages = (1 << 32) // (heads * ps * hd // 2) + 40
    S = torch.tensor([0.01, 0.02], device=DEV)
    cache = kvcache.KVCache.empty(pages, ps, heads, hd, S, S)
    n = 700
    k, v = _kv(71, BF, n, heads, hd)
    page = torch.tensor([pages - 1, pages - 3], dtype=torch.int64)
    slots = page[torch.arange(n) // ps] * ps + torch.arange(n) % ps
    kvcache.write(cache, strided(k), strided(v), slots.to(DEV))
    small = kvcache.KVCache.empty(2, ps, heads, hd, S, S)
    kvcache.write(small, strided(k), strided(v), torch.arange(n, device=DEV))
    for a, b in zip(kvcache.read(cache, slots.to(DEV), F32), kvcache.read(small, torch.arange(n, device=DEV), F32)):
        assert torch.equal(a, b)
    q = torch.randn(1, 8, hd, device=DEV).to(BF)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    a = kvcache.attention(cache, q, page.int().view(1, 2).to(DEV), lens)
    b = kvcache.attention(small, q, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), lens)
    assert torch.equal(a, b)


def test_empty_calls():
    case("kv calls with nothing to do")
    S = torch.ones(2, device=DEV)
    cache = kvcache.KVCache.empty(2, 16, 2, 64, S, S)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    kvcache.write(cache, torch.empty(0, 2, 64, device=DEV), torch.empty(0, 2, 64, device=DEV), none)
    assert kvcache.read(cache, none)[0].shape == (0, 2, 64)
    q = torch.empty(0, 4, 64, device=DEV, dtype=BF)
    assert kvcache.attention(cache, q).shape == (0, 4, 64)
    # no pages at all: every query sees nothing
    cache = kvcache.KVCache.empty(0, 16, 2, 64, S, S)
    q = torch.randn(3, 4, 64, device=DEV)
    out, lse = kvcache.attention(cache, q, torch.zeros(3, 2, dtype=torch.int32, device=DEV),
                                 torch.full((3,), 9, dtype=torch.int32, device=DEV), return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = kvcache.attention(cache, q, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert (kvcache.read(cache, torch.tensor([0, 5], device=DEV))[0] == 0).all()


def test_debug_checks_see_the_new_inputs(monkeypatch):
    case("kv write with debug checks on")
    monkeypatch.setenv("NVFP4_DEBUG_CHECKS", "1")
    S = torch.ones(2, device=DEV)
    cache = kvcache.KVCache.empty(2, 16, 2, 64, S, S)
    k = torch.zeros(3, 2, 64, device=DEV)
    slots = torch.arange(3, device=DEV)
    nvfp4.debug_nonfinite()
    kvcache.write(cache, k, k, slots)
    assert not nvfp4.debug_nonfinite()
    v = k.clone()
    v[1, 1, 7] = math.inf
    kvcache.write(cache, k, v, slots)
    assert nvfp4.debug_nonfinite()
    kvcache.attention(cache, v)
    assert nvfp4.debug_nonfinite()
    assert not nvfp4.debug_nonfinite()
