"""The attention's kernel variants and plans, each reached on purpose, with the references and the
bounds of test_gpu_kvcache.py: row counts around every change of kernel, contexts cut into pieces
and whole, contexts of several page runs, more sequences than a wave has lanes, prefixes in the
same launch and in their own, loose bounds, shared workspaces."""
import numpy as np
import pytest
import torch

import kvcache_ref as ref
from scale_search_weights_amd import kvcache
from test_gpu_kvcache import BF, DEV, F32, attend, case, check, on_gpu, strided
from test_gpu_kvcache import test_write_matches_the_quantiser_and_read_dequantises as write_and_read

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [15, 16, 17, 32, 33, 64, 65, 128, 129, 300])
def test_rows_a_head(dtype, hd, rows):
    """Rows a (sequence, key/value head) around 16, 32, 64, 128 and 256."""
    case(f"kv attention, {rows} rows a head of {hd}, {dtype}")
    c = ref.make(rows + hd, dtype, [rows, max(1, rows // 3)], [rows + 70, rows // 3 + 40], 2, 2, hd, 16, 45)
    check(c, attend(c))


@pytest.mark.parametrize("rows,kv,hd,dtype", [
    (600, 2500, 128, BF), (600, 2500, 64, BF), (300, 1300, 256, BF), (300, 1300, 128, F32),   # several page runs
    (80, 2600, 128, BF), (40, 2600, 64, BF), (40, 2100, 256, F32)])                          # cut into pieces
def test_long_contexts_with_many_rows(rows, kv, hd, dtype):
    case(f"kv attention, {rows} queries on {kv} tokens, head_dim {hd}, {dtype}")
    c = ref.make(rows + kv, dtype, [rows], [kv], 2, 1, hd, 32)
    check(c, attend(c))


@pytest.mark.parametrize("batch,kv,heads,kv_heads,hd,page_size", [
    (1, 1500, 4, 2, 128, 16),     # whole, sixteen waves
    (1, 1600, 4, 2, 128, 512),    # in pieces
    (40, 700, 16, 8, 64, 16),     # whole, eight waves
    (70, 300, 16, 8, 128, 16),    # whole, four waves, more sequences than a wave's lanes
    (150, 420, 2, 1, 128, 16),    # sequences in three lane groups
    (130, 2100, 4, 2, 64, 64),    # in pieces, sequences in three lane groups
])
def test_batches(batch, kv, heads, kv_heads, hd, page_size):
    case(f"kv attention, {batch} sequences of up to {kv} tokens")
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, kv + 1, batch)]
    lens[0], lens[-1] = kv, 0
    if batch > 2:
        lens[batch // 2] = 1
    c = ref.make(batch, BF, [1] * batch, lens, heads, kv_heads, hd, page_size)
    check(c, attend(c))


@pytest.mark.parametrize("q_lens,lens,prefix,heads,kv_heads,hd,dtype", [
    ([1] * 9, [30, 0, 200, 7, 1, 90, 128, 129, 300], 1200, 8, 2, 128, BF),   # prefix apart, many rows
    ([1] * 3, [30, 0, 200], 60, 8, 2, 128, BF),                              # one launch
    ([40, 3], [90, 3], 700, 4, 2, 64, BF),                                   # both with many rows
    ([40, 3], [90, 3], 20, 4, 2, 128, BF),
    ([2, 1], [1900, 40], 300, 8, 2, 256, F32),                               # own tokens in pieces, prefix too
    ([1, 1], [1900, 1400], 900, 6, 1, 128, BF),
    ([0, 0, 5], [50, 0, 5], 130, 3, 3, 96, BF),
])
def test_prefix_and_own_tokens(q_lens, lens, prefix, heads, kv_heads, hd, dtype):
    for causal in (True, False):
        case(f"kv attention, prefix {prefix}, own {lens}, queries {q_lens}, causal {causal}")
        c = ref.make(sum(lens) + prefix, dtype, q_lens, lens, heads, kv_heads, hd, 16, prefix)
        check(c, attend(c, causal=causal), causal)


def test_prefix_alone():
    """No own tokens at all: no block table; short (written at once) and in pieces."""
    for prefix in (40, 3000):
        case(f"kv attention over a prefix of {prefix} alone")
        c = ref.make(prefix, BF, [1, 2, 1], [0, 0, 0], 8, 2, 128, 16, prefix)
        check(c, attend(c))


def test_loose_query_bound_with_a_prefix():
    """max_q left at the token count: rows that belong to no sequence's bound stay out."""
    case("kv attention with max_q = tokens")
    c = ref.make(5, BF, [9, 0, 30, 2], [20, 5, 64, 130], 8, 2, 64, 16, 77)
    check(c, attend(dict(c, max_q=41)))
    c = ref.make(6, BF, [1, 1, 1], [900, 5, 640], 8, 2, 64, 16)
    check(c, attend(dict(c, max_q=3)))


def test_workspace_of_the_caller():
    """A given workspace, dirty, reused by calls of other shapes; out given too."""
    case("kv attention with the caller's workspace and out")
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    for seed, q_lens, lens, prefix in ((1, [1] * 5, [700, 0, 3000, 5, 64], 0), (2, [1] * 30, [100] * 30, 900),
                                       (3, [3, 1], [2500, 80], 60)):
        c = ref.make(seed, BF, q_lens, lens, 8, 2, 128, 16, prefix)
        want = attend(c)
        q = strided(c["q"])
        out = torch.full(c["q"].shape, float("nan"), dtype=BF, device=DEV)
        got = kvcache.attention(on_gpu(c), q, c["table"].to(DEV), c["kv_lens"].to(DEV),
                                q_offsets=c["q_offsets"].to(DEV), max_q=c["max_q"], max_kv=c["max_kv"],
                                prefix_pages=c["prefix_pages"].to(DEV) if prefix else None, prefix_len=prefix,
                                out=out, workspace=ws)
        assert got is out and torch.equal(out, want[0])
        check(c, want)


def test_lengths_of_one_to_forty():
    """Every length around the 16- and 32-token groups, one new token and all queries at once."""
    case("kv attention, lengths 1 to 40")
    lens = list(range(1, 41))
    c = ref.make(8, BF, [1] * 40, lens, 4, 2, 64, 16)
    check(c, attend(c))
    c = ref.make(9, BF, lens, lens, 4, 1, 128, 16)
    check(c, attend(c))
    check(c, attend(c, causal=False), causal=False)


def test_page_runs_and_pages_larger_than_a_run():
    """Pages of 32768 tokens, and contexts whose last run holds one token."""
    for n, ps in ((2049, 16), (1025, 32768), (4097, 64)):
        case(f"kv attention, {n} tokens in pages of {ps}")
        c = ref.make(n, BF, [1], [n], 2, 1, 64, ps, spare_pages=1)
        check(c, attend(c))
        c = ref.make(n, BF, [50], [n], 2, 1, 64, ps, spare_pages=1)
        check(c, attend(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd", [64, 80, 128, 144, 256])
@pytest.mark.parametrize("rows", [50, 100, 150, 280])
def test_large_calls(dtype, hd, rows):
    """Calls of over 512 workgroups, whose tiles are larger: rows in one, two and more tiles,
    contexts of unequal lengths, one of them empty; the second call over a prefix alone and own tokens."""
    case(f"kv attention, {rows} rows a head of {hd}, {dtype}, many workgroups")
    q = rows // 2
    lens = [1030, 1030 - q, 0, 517, 130, 1029, 800, 31]
    c = ref.make(rows + hd, dtype, [q, q - 1, 0, 3, q, 1, q // 2, 31 % (q + 1)], lens, 16, 8, hd, 32)
    check(c, attend(c))
    c = ref.make(rows + hd + 1, dtype, [rows // 4, 1, rows // 4 - 1], [rows // 4, 300, 40], 16, 8, hd, 32, 8200)
    check(c, attend(c))


@pytest.mark.parametrize("dtype,tokens,heads,hd,page_size", [
    (BF, 4999, 4, 112, 32), (F32, 4999, 4, 112, 32),        # several rows a lane, an odd count of tokens
    (BF, 40003, 4, 16, 16), (F32, 2051, 1, 1024, 64)])      # the smallest and the largest rows
def test_write_and_read_of_many_tokens(dtype, tokens, heads, hd, page_size):
    write_and_read(dtype, tokens, heads, hd, page_size, None, False)


def test_refuses_a_cache_that_is_not_on_the_current_device():
    """Kernels are launched on the current device: a cache of another one is refused, not read."""
    case("kv cache on another device than the current one")
    c = ref.make(4, BF, [1], [20], 2, 1, 64, 16)
    cache = on_gpu(c)
    cache._index += 1  # as if the current device had been changed
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    k = torch.zeros(1, 1, 64, dtype=BF, device=DEV)
    for call in (lambda: attend(c, cache), lambda: kvcache.read(cache, slots),
                 lambda: kvcache.write(cache, k, k, slots)):
        with pytest.raises(ValueError, match="current device"):
            call()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd,prefix,causal", [(64, 700, True), (128, 77, True), (128, 129, False), (112, 1, True),
                                              (256, 300, True), (144, 2100, True)])
def test_prefix_before_own_tokens_in_one_workgroup(dtype, hd, prefix, causal):
    """Sequences that fill tiles of their own go over the prefix first: large and small calls,
    sequences without own tokens, without queries, with a hidden page in the prefix."""
    case(f"kv attention, prefix {prefix} before own tokens, head_dim {hd}, {dtype}, causal {causal}")
    q = [280, 279, 0, 3, 280, 1, 140, 31]
    c = ref.make(prefix + hd, dtype, q, [1030, 750, 0, 517, 300, 1029, 800, 0], 16, 8, hd, 32, prefix)
    check(c, attend(c, causal=causal), causal)
    c = ref.make(prefix + hd + 1, dtype, [128, 5, 100], [128, 0, 110], 4, 2, hd, 16, prefix)
    check(c, attend(c, causal=causal), causal)
    if prefix > 200:
        c["prefix_pages"][3] = -1
        check(c, attend(c, causal=causal), causal)
