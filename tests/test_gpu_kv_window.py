"""Windowed attention with sinks on the GPU against 64 bits (kv_window_ref.py)."""
import pytest
import torch

import kv_window_ref as win
import kvcache_ref as ref
from scale_search_weights_amd import kvcache
from test_gpu_kvcache import on_gpu, strided

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def case(msg):
    print(f"[case] {msg}", flush=True)


def attend(c, window, sinks, cache=None, scale=None, **kw):
    return kvcache.attention(cache or on_gpu(c), strided(c["q"]), c["table"].to(DEV), c["kv_lens"].to(DEV),
                             q_offsets=c["q_offsets"].to(DEV), max_q=c["max_q"], max_kv=c["max_kv"], window=window,
                             sinks=sinks, scale=scale, return_lse=True, **kw)


SHAPES = [
    # dtype, q_lens, kv_lens, heads, kv_heads, hd, page_size, window, sinks
    (BF, [1], [1], 1, 1, 64, 16, 1, 0),
    (BF, [1], [1000], 32, 8, 128, 16, 512, 4),
    (BF, [1] * 6, [17, 0, 300, 16, 129, 48], 8, 2, 128, 16, 16, 0),
    (BF, [1] * 6, [17, 0, 300, 16, 129, 48], 8, 2, 128, 16, 1, 1),
    (BF, [1] * 6, [17, 0, 300, 16, 129, 48], 8, 2, 64, 16, 33, 17),
    (BF, [1] * 4, [40, 2, 31, 700], 16, 2, 128, 32, 100, 15),
    (BF, [1] * 4, [40, 2, 31, 700], 16, 2, 128, 32, 100, 16),
    (BF, [1] * 4, [40, 2, 31, 700], 16, 2, 128, 32, 100, 600),   # sinks reach the window
    (BF, [1] * 4, [40, 2, 31, 700], 16, 2, 128, 32, 5000, 3),    # the window covers everything
    (BF, [1] * 4, [40, 2, 31, 700], 16, 2, 128, 32, 1 << 30, 1 << 30),
    (BF, [3, 0, 5, 1], [3, 0, 900, 64], 12, 4, 128, 64, 50, 2),
    (BF, [4, 2], [2, 300], 4, 1, 96, 16, 20, 3),                 # more queries than cached tokens
    (BF, [8, 9], [1500, 2700], 4, 2, 128, 16, 1200, 4),          # 16 and 18 rows, in pieces
    (BF, [7, 9, 40], [100, 9, 333], 28, 4, 128, 16, 64, 4),
    (BF, [130], [130], 6, 2, 128, 16, 32, 1),
    (BF, [70, 200], [500, 200], 8, 2, 64, 32, 77, 19),
    (BF, [300, 1, 0, 40], [900, 1, 50, 40], 8, 8, 128, 16, 128, 4),
    (BF, [33, 65], [150, 90], 10, 5, 80, 16, 40, 5),
    (BF, [1] * 40, [100] * 39 + [2], 8, 2, 128, 16, 30, 4),
    (BF, [5], [200], 8, 1, 256, 16, 60, 5),
    (BF, [100], [260], 4, 2, 256, 128, 48, 0),
    (BF, [6], [90], 3, 3, 16, 16, 20, 2),
    (BF, [37], [90], 4, 2, 160, 16, 20, 2),
    (BF, [600], [3000], 4, 2, 128, 64, 1000, 100),
    (F32, [1], [333], 8, 2, 128, 16, 64, 4),
    (F32, [4, 1, 3], [400, 0, 77], 8, 1, 256, 16, 65, 5),
    (F32, [50, 90], [180, 90], 6, 2, 64, 16, 31, 2),
    (F32, [300], [420], 4, 1, 128, 64, 100, 20),
    (F32, [20], [80], 5, 5, 112, 16, 7, 0),
    (F32, [4, 2], [4001, 2500], 8, 1, 256, 16, 777, 5),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_window(shape):
    dtype, q_lens, kv_lens, heads, kv_heads, hd, ps, window, sinks = shape
    case(f"kv window {shape}")
    c = ref.make(len(q_lens) * 100 + hd, dtype, q_lens, kv_lens, heads, kv_heads, hd, ps)
    win.check(c, attend(c, window, sinks), window, sinks)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 112, 127, 128, 129, 130, 144])
def test_every_offset_of_window_and_length(window):
    """Contexts of every length mod 16 around the window's, sinks around a group of 16: decoding, and a few
    rows whose windows differ."""
    case(f"kv window {window} at every offset")
    for sinks in (0, 1, 15, 16, 17):
        kv = list(range(max(1, window + sinks - 9), window + sinks + 40))
        c = ref.make(window * 100 + sinks, BF, [1 + b % 3 for b in range(len(kv))], kv, 4, 2, 64, 16)
        win.check(c, attend(c, window, sinks), window, sinks)


def test_long_context_costs_and_gives_the_window():
    case("kv window: 40000 tokens")
    c = ref.make(1, BF, [1, 2], [40000, 39990], 6, 2, 128, 64)
    win.check(c, attend(c, 4096, 128), 4096, 128)
    win.check(c, attend(c, 1, 0), 1, 0)


def test_evicted_pages():
    """Pages between the sinks and the window are gone: any id, and pages that other sequences own now."""
    case("kv window: evicted pages")
    c = ref.make(3, BF, [1, 3, 20], [500, 700, 333], 8, 2, 128, 16)
    window, sinks = 100, 20
    want = attend(c, window, sinks)
    for b, (n, m) in enumerate(((1, 500), (3, 700), (20, 333))):
        t = win.seen(n, m, window, sinks).any(0)
        for page in range(-(-m // 16)):
            if not t[16 * page:16 * page + 16].any():
                c["table"][b, page] = (-1, 1 << 30, -(1 << 31), 0, 5)[page % 5]
    got = attend(c, window, sinks)
    win.check(c, got, window, sinks)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_pages_in_sight_are_hidden():
    case("kv window: bad page ids among the seen")
    c = ref.make(4, BF, [1, 2, 40], [300, 60, 200], 8, 2, 64, 16)
    c["table"][0, 0], c["table"][0, 17], c["table"][1, 3], c["table"][2, 11] = -1, 1 << 20, -7, 1 << 30
    c["table"][1, :] = -1
    win.check(c, attend(c, 50, 3), 50, 3)


def test_a_window_of_everything_is_full_attention():
    case("kv window against full attention")
    c = ref.make(5, F32, [5, 1, 60], [50, 700, 200], 8, 2, 128, 16)
    full = kvcache.attention(on_gpu(c), strided(c["q"]), c["table"].to(DEV), c["kv_lens"].to(DEV),
                             q_offsets=c["q_offsets"].to(DEV), max_q=60, max_kv=700, return_lse=True)
    got = attend(c, 700, 0)
    win.check(c, got, 700, 0)
    win.check(c, full, 700, 0)


@pytest.mark.parametrize("dtype,qs,scale", [(BF, 40.0, None), (F32, 40.0, None), (BF, 1e30, 1e-30), (BF, 1.0, 0.0),
                                            (BF, 1.0, -0.2), (F32, 1e-20, 1e20)])
def test_large_scores_and_scales(dtype, qs, scale):
    case(f"kv window, q ~ {qs}, scale {scale}, {dtype}")
    c = ref.make(9, dtype, [2, 1, 50], [210, 64, 90], 8, 2, 128, 16, q_scale=qs)
    win.check(c, attend(c, 40, 4, scale=scale), 40, 4, scale=scale)


def test_queries_that_are_not_finite():
    case("kv window: NaN and infinite queries")
    c = ref.make(10, BF, [3, 40], [900, 300], 8, 2, 64, 16)
    good, clean = dict(c, q=c["q"].clone()), attend(c, 64, 4)
    bad = torch.zeros(43, 8, dtype=torch.bool)
    for t, h, x in ((0, 1, float("nan")), (2, 7, float("inf")), (17, 0, float("-inf")), (42, 5, float("nan"))):
        c["q"][t, h, 11], bad[t, h] = x, True
    out, lse = attend(c, 64, 4)
    bad = bad.to(DEV)
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    # The rows beside them stay within the bounds. Not bit for bit: a row that never fits fp16's range has
    # its whole wave take a new maximum in every tile, which rounds the other rows' sums elsewhere.
    win.check(good, (torch.where(bad.unsqueeze(-1), clean[0], out), torch.where(bad, clean[1], lse)), 64, 4)


def test_loose_bounds_lengths_past_them_and_rows_of_no_sequence():
    case("kv window: loose max_q and max_kv, lengths over and under them")
    c = ref.make(11, BF, [2, 1, 3], [100, 50, 260], 4, 2, 64, 16)
    want = attend(c, 30, 4)
    c2 = dict(c, max_q=6, max_kv=272)
    assert all(torch.equal(a, b) for a, b in zip(attend(c2, 30, 4), want))
    short = dict(c, max_kv=90, kv_lens=torch.tensor([100, -5, 1 << 30], dtype=torch.int32))
    got = attend(short, 30, 4)
    win.check(dict(c, kv_lens=torch.tensor([90, 0, 90])), got, 30, 4)
    out = torch.full((6, 4, 64), 7.0, dtype=BF, device=DEV)
    part = dict(c, q_offsets=torch.tensor([1, 3, 4, 6], dtype=torch.int32))
    attend(part, 30, 4, out=out)
    assert (out[0] == 7).all()  # this row belongs to no sequence and nothing was written there


def test_side_stream_graph_workspace():
    case("kv window: side stream, graphs that share a workspace, poisoned workspaces")
    c = ref.make(12, BF, [1] * 3, [3000, 2000, 100], 8, 2, 128, 16)
    cache, q = on_gpu(c), strided(c["q"])
    table, lens = c["table"].to(DEV), c["kv_lens"].to(DEV)
    need = kvcache.attention_workspace_size(cache, BF, 3, 8, 3, 1, 3000, window=1500, sinks=4)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)

    def call(window):
        return kvcache.attention(cache, q, table, lens, max_kv=3000, window=window, sinks=4, workspace=ws)
    want = {w: call(w).clone() for w in (1500, 1200)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(call(1500), want[1500])
    torch.cuda.current_stream().wait_stream(side)
    graphs = {}
    for w in (1500, 1200):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(w)
        graphs[w] = (g, out)
    for step in range(4):
        ws.fill_(step * 85)
        for w, (g, out) in graphs.items():
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[w])
        assert torch.equal(call(1500), want[1500])
    win.check(c, attend(c, 1500, 4), 1500, 4)


def test_slots_past_32_bits():
    case("kv window: pages beyond 2^31 bytes")
    c = ref.make(13, BF, [1, 40], [600, 700], 4, 2, 64, 1024)
    kc, ks, vc, vs, S_k, S_v, _ = c["cache"]
    n, far = kc.shape[0], 1 << 15
    big = kvcache.KVCache.empty(far + n, 1024, 2, 64, S_k.to(DEV), S_v.to(DEV))
    for t, x in ((big.k_codes, kc), (big.k_scales, ks), (big.v_codes, vc), (big.v_scales, vs)):
        t[far:].copy_(x)
    want = attend(c, 200, 10)
    c["table"] += far
    got = attend(c, 200, 10, cache=big)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
