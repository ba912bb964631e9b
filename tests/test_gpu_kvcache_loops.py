"""write and read of more rows than one pass of their grid takes: the later iterations of both kernels."""
import pytest
import torch

from scale_search_weights_amd import kvcache, nvfp4
from test_gpu_kvcache import BF, DEV, F32, case

pytestmark = pytest.mark.gpu


def _by_head(x, slots, page_size, want, bytes_of):
    """Put bytes_of(head) into the slots of `want`, head by head."""
    keep = slots >= 0
    page, at = slots[keep] // page_size, slots[keep] % page_size
    for h in range(want.shape[1]):
        want[page, h, at] = bytes_of(h)[keep]


@pytest.mark.parametrize("tokens,heads,hd,page_size", [
    (601, 520, 1024, 32),          # 64 chunks of 8 tokens a head, the smallest grid, and 11 more
    (5_700_001, 3, 16, 128)])      # over 10922 chunks of 512 tokens of 3 heads
def test_more_chunks_than_the_grid(tokens, heads, hd, page_size):
    case(f"kv write/read of {tokens} tokens of {heads} heads of {hd}")
    g = torch.Generator(device=DEV).manual_seed(tokens)
    kv = [(torch.randn(tokens, heads, hd, generator=g, device=DEV) * 3).to(BF) for _ in range(2)]
    S = torch.rand(heads, generator=g, device=DEV) * 0.004 + 0.001
    pages = -(-tokens // page_size) + 1
    slots = torch.randperm(pages * page_size, generator=g, device=DEV)[:tokens]
    slots[torch.rand(tokens, generator=g, device=DEV) < 0.1] = -1
    slots[[0, tokens // 2, tokens - 2]] = -1
    cache = kvcache.KVCache.empty(pages, page_size, heads, hd, S, S)
    stores = ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))
    for c, s in stores:
        c.fill_(0xA5), s.fill_(0x5A)
    kvcache.write(cache, *kv, slots)
    dense = []
    for x, (c, s) in zip(kv, stores):
        packed = [nvfp4.quantize(x[:, h].contiguous(), S[h:h + 1]) for h in range(heads)]
        for got, n, fill in ((c, 0, 0xA5), (s, 1, 0x5A)):
            want = torch.full_like(got, fill)
            _by_head(x, slots, page_size, want, lambda h: packed[h][n])
            assert torch.equal(got, want)
            del want
        dense.append(packed)
    hidden = (slots < 0).view(-1, 1)
    for dtype in (BF, F32):
        for y, packed in zip(kvcache.read(cache, slots, dtype), dense):
            for h in range(heads):
                want = nvfp4.dequantize(*packed[h], S[h:h + 1], dtype)
                assert torch.equal(y[:, h], want.masked_fill(hidden, 0)), h
