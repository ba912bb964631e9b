"""Append with the rotation on the way: cache bytes and turned queries, bit for bit those of the rotation
(test_gpu_rotary.py) followed by the library's quantiser."""
import numpy as np
import pytest
import torch

import kvcache_ref as ref
from scale_search_weights_amd import kvcache, nvfp4, rotary
from test_gpu_kvcache import _kv, strided

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def case(msg):
    print(f"[case] {msg}", flush=True)


def turn(rng, hd, pairs, axes, adjacent, factor, tokens):
    w = torch.from_numpy(1e4 ** (-np.arange(pairs) / pairs)).to(DEV)
    axis = torch.from_numpy(rng.integers(0, axes, pairs).astype(np.int32)).to(DEV) if axes > 1 else None
    pos = torch.from_numpy(rng.integers(0, 200000, (axes, tokens))).to(DEV)
    return rotary.Rotary(w, axis, axes=axes, adjacent=adjacent, factor=factor), pos


def expected(before, k, v, slots, S_k, S_v, rot, pos):
    """The cache's tensors after an append to `before`."""
    kt = rotary.rotate(k.to(DEV).float(), pos, rot)
    out = [t.clone() for t in before]
    pages, heads, size, _ = out[0].shape
    keep = ((slots >= 0) & (slots < pages * size)).nonzero().squeeze(1)
    at = slots[keep]
    for n, x, S in ((0, kt, S_k), (2, v.to(DEV), S_v)):
        for h in range(heads):
            c, s = nvfp4.quantize(x[:, h].contiguous(), S[h:h + 1].to(DEV))
            out[n][at // size, h, at % size] = c.cpu()[keep]
            out[n + 1][at // size, h, at % size] = s.cpu()[keep]
    return out


SHAPES = [
    # dtype, tokens, heads, kv_heads, head_dim, pairs, page, axes, adjacent, factor, ties
    (BF, 1, 4, 1, 128, 64, 16, 1, False, 1.0, False), (BF, 48, 32, 8, 128, 64, 16, 1, False, 1.0, False),
    (F32, 101, 10, 5, 80, 40, 32, 1, False, 1.0, False), (BF, 257, 6, 3, 64, 32, 64, 3, False, 1.0, False),
    (F32, 130, 4, 2, 256, 128, 16, 1, True, 1.0, True), (BF, 70, 0, 4, 96, 24, 128, 2, True, 1.25, True),
    (F32, 19, 2, 1, 1024, 512, 16, 1, False, 1.0, False), (BF, 21, 4, 2, 1008, 8, 16, 16, False, 1.0, False),
    (BF, 3000, 7, 1, 112, 56, 256, 1, False, 0.875, False), (BF, 40, 3, 3, 16, 8, 16, 1, False, 1.0, False),
    (F32, 33, 0, 2, 48, 16, 16, 1, True, 1.0, False), (BF, 700, 28, 4, 128, 32, 64, 3, False, 1.0, False)]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_append(shape):
    dtype, tokens, heads, kv_heads, hd, pairs, page, axes, adjacent, factor, ties = shape
    case(f"kv append {shape}")
    rng = np.random.default_rng(hd + tokens)
    k, v = _kv(tokens + hd, dtype, tokens, kv_heads, hd, ties)
    rot, pos = turn(rng, hd, pairs, axes, adjacent, factor, tokens)
    pages = -(-tokens // page) + 1
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int64))
    slots[torch.from_numpy(rng.random(tokens) < 0.15)] = -1
    if tokens > 3:
        slots[1], slots[2], slots[3] = pages * page, -(1 << 62), 1 << 62
    S_k = (k.float().abs().amax((0, 2)) / 2688).clamp(min=1e-6) if not ties else torch.full((kv_heads,), 1 / 512)
    S_v = (v.float().abs().amax((0, 2)) / 2688).clamp(min=1e-6)
    before = [ref.any_bytes(rng, (pages, kv_heads, page, n)) for n in (hd // 2, hd // 16) * 2]
    cache = kvcache.KVCache(*(t.to(DEV) for t in before), S_k.to(DEV), S_v.to(DEV))
    q = torch.from_numpy(rng.standard_normal((tokens, heads + 1, hd)).astype(np.float32)).to(dtype)[:, :heads]
    qg = strided(q)
    got = kvcache.append(cache, strided(k), strided(v), slots.to(DEV), pos, rot, q=qg if heads else None)
    want = expected(before, k, v, slots, S_k, S_v, rot, pos)
    for name, a, b in zip(("k codes", "k scales", "v codes", "v scales"),
                          (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), want):
        assert torch.equal(a.cpu(), b), name
    if heads:
        assert torch.equal(got, rotary.rotate(qg, pos, rot))
    else:
        assert got is None


def _small(seed=0, tokens=40, dtype=BF, heads=4, kv_heads=2, hd=64, pairs=32, page=16, pages=4):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((tokens, heads + 2 * kv_heads, hd)).astype(np.float32)).to(dtype).to(DEV)
    rot, pos = turn(rng, hd, pairs, 1, False, 1.0, tokens)
    S = torch.full((kv_heads,), 6.0 / 2688, device=DEV)
    cache = kvcache.KVCache.empty(pages, page, kv_heads, hd, S, S)
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens]).to(DEV)
    return cache, qkv, rot, pos, slots


def _bytes(cache, slots):
    return [t[slots // cache.page_size, :, slots % cache.page_size].clone()
            for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def test_queries_in_place_and_values_as_write_has_them():
    case("kv append: queries in place in the fused rows; values as write")
    cache, qkv, rot, pos, slots = _small()
    want_q = rotary.rotate(qkv[:, :4], pos, rot)
    k, v = qkv[:, 4:6].clone(), qkv[:, 6:].clone()
    q = qkv[:, :4]
    assert kvcache.append(cache, qkv[:, 4:6], qkv[:, 6:], slots, pos, rot, q=q, q_out=q) is q
    assert torch.equal(q, want_q) and torch.equal(qkv[:, 4:6], k) and torch.equal(qkv[:, 6:], v)
    got = _bytes(cache, slots)
    kvcache.write(cache, k, v, slots)
    assert all(torch.equal(a, b) for a, b in zip(got[2:], _bytes(cache, slots)[2:]))
    # at position 0 nothing turns, and append is write
    kvcache.append(cache, k, v, slots, torch.zeros_like(pos), rot)
    now = _bytes(cache, slots)
    kvcache.write(cache, k, v, slots)
    assert all(torch.equal(a, b) for a, b in zip(now, _bytes(cache, slots)))


def test_no_tokens_no_pages_no_heads():
    case("kv append with nothing to store")
    cache, qkv, rot, pos, slots = _small()
    before = [t.clone() for t in (cache.k_codes, cache.v_scales)]
    none = kvcache.append(cache, qkv[:0, 4:6], qkv[:0, 6:], slots[:0], pos[:, :0], rot, q=qkv[:0, :4])
    assert none.shape == (0, 4, 64)
    kvcache.append(cache, qkv[:, 4:6], qkv[:, 6:], torch.full_like(slots, -1), pos, rot)
    assert torch.equal(before[0], cache.k_codes) and torch.equal(before[1], cache.v_scales)
    empty = kvcache.KVCache.empty(0, 16, 2, 64, cache.S_k, cache.S_v)
    q = kvcache.append(empty, qkv[:, 4:6], qkv[:, 6:], slots, pos, rot, q=qkv[:, :4])
    assert torch.equal(q, rotary.rotate(qkv[:, :4], pos, rot))


def test_slots_past_32_bits():
    case("kv append: slots beyond 2^31 bytes")
    cache, qkv, rot, pos, slots = _small()
    big = kvcache.KVCache.empty(1 << 15, 1024, 2, 64, cache.S_k, cache.S_v)  # 2 GiB of key codes
    far = (1 << 25) - 1 - torch.arange(40, device=DEV)
    kvcache.append(big, qkv[:, 4:6], qkv[:, 6:], far, pos, rot)
    kvcache.append(cache, qkv[:, 4:6], qkv[:, 6:], slots, pos, rot)
    assert all(torch.equal(a, b) for a, b in zip(_bytes(big, far), _bytes(cache, slots)))


def test_graph_of_decoding_steps():
    """A captured step (append, then attention over what it wrote) replayed with new inputs."""
    case("kv append and attention in a graph")
    cache, qkv, rot, pos, _ = _small(tokens=4, pages=8, page=16)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    lens = torch.zeros(4, dtype=torch.int32, device=DEV)
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)

    def step():
        q = kvcache.append(cache, qkv[:, 4:6], qkv[:, 6:], slots, pos, rot, q=qkv[:, :4])
        return kvcache.attention(cache, q, table, lens, max_kv=32, window=7, sinks=2)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = torch.Generator(device=DEV).manual_seed(3)
    for n in range(20):
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV))
        pos.fill_(n)
        lens.fill_(n + 1)
        slots.copy_(table[:, n // 16].long() * 16 + n % 16)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
