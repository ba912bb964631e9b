"""Rotary positions, append to the NVFP4 key/value cache and attention over a window of it, as measured work.

Three operators around an attention layer whose keys and values are cached in NVFP4 (E2M1 codes,
one E4M3 scale per 16 values along the head dimension, one fp32 scale per head):

* ``rotate``  rotary positions of one or several axes (time, height, width), with gradients;
* ``append``  rotates new keys on the way into the cache, stores the values beside them and rotates
              the step's queries; the written slots are read back;
* ``window``  softmax attention of new queries over a sliding window of the cached tokens and
              over the first tokens, which stay visible (sinks).

With ``own`` false, ``run`` is elementary torch in fp32 (angles in fp64); with ``own`` true it
calls ``scale_search_weights_amd.rotary`` and ``scale_search_weights_amd.kvcache``.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
# sections: the pairs of each axis in order, as text; their sum is half the rotated channels.
# place: how positions come about (_positions).

def _rotate(name, dtype, tokens, heads, head_dim, sections, place, base=10000.0, adjacent=False,
            factor=1.0, train=False):
    return {"name": name, "op": "rotate", "dtype": dtype, "tokens": tokens, "heads": heads,
            "head_dim": head_dim, "sections": sections, "place": place, "base": base,
            "adjacent": adjacent, "factor": factor, "train": train}


def _append(name, dtype, tokens, heads, kv_heads, head_dim, page_size, sections, place, base=10000.0,
            adjacent=False, factor=1.0, skipped=False):
    return {"name": name, "op": "append", "dtype": dtype, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page_size": page_size, "sections": sections,
            "place": place, "base": base, "adjacent": adjacent, "factor": factor, "skipped": skipped}


def _window(name, dtype, batch, q_len, heads, kv_heads, head_dim, page_size, kv_len, window, sinks,
            ragged=False):
    return {"name": name, "op": "window", "dtype": dtype, "batch": batch, "q_len": q_len,
            "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page_size": page_size,
            "kv_len": kv_len, "window": window, "sinks": sinks, "ragged": ragged}


def listed():
    return [
        # queries and keys of one decoding step of 32 sequences
        _rotate("rotate_step", "bf16", 32, 40, 128, "64", "step"),
        # a video in a prompt: time, height and width, queries and keys of one fused projection
        _rotate("rotate_video", "bf16", 12000, 32, 128, "16,24,24", "video", base=1e6),
        # training an image encoder in fp32, heads of 72 channels, patch rows and columns; forward
        # and backward
        _rotate("rotate_train", "fp32", 9801, 16, 72, "18,18", "image", train=True),
        # one decoding step: a new token of each of 48 sequences
        _append("append_step", "bf16", 48, 32, 8, 128, 16, "64", "step"),
        # prompts of a batch packed to 16384 tokens, far into a long context
        _append("append_prompt", "bf16", 16384, 32, 8, 128, 64, "64", "text", base=1e6),
        # a prompt with images and video, stretched context (cosines and sines times a factor)
        _append("append_video", "bf16", 7001, 28, 4, 128, 64, "16,24,24", "video", base=1e6, factor=1.2),
        # fp32 model, head size 80 of which 48 channels turn in adjacent pairs, a padded batch
        _append("append_padded_fp32", "fp32", 5003, 10, 5, 80, 32, "24", "text", adjacent=True,
                skipped=True),
        # one user behind a thousand tokens, a short window: the smallest step
        _window("window_one", "bf16", 1, 1, 32, 8, 128, 16, 1000, 512, 4),
        # a decoding batch of unequal lengths (one slot of the batch idle)
        _window("window_batch", "bf16", 64, 1, 32, 8, 128, 32, 8192, 1024, 4, ragged=True),
        # few sequences, very long context, a window of some thousand tokens
        _window("window_long", "bf16", 4, 1, 64, 8, 64, 64, 131000, 4096, 128),
        # a prompt chunk of two sequences over what is cached of them
        _window("window_prompt", "bf16", 2, 2048, 32, 8, 128, 64, 8192, 1024, 16),
        # fp32, wide heads with one key/value head, a few drafted tokens to be verified
        _window("window_draft_fp32", "fp32", 7, 4, 8, 1, 256, 16, 4001, 777, 5, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_BYTES, MOST_FLOPS = 3.5e8, 6.9e10  # of the largest listed cases


def _split_pairs(rng, pairs, axes):
    """Sections of the pairs over the axes, none empty."""
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(("rotate", "append", "window", "window"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op == "window":
        head_dim = rng.choice((64, 64, 80, 96, 128, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 5, 8))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
        kind = rng.choice(("step", "step", "draft", "prompt"))
        window, sinks = _log_int(rng, 16, 8192), rng.choice((0, 1, 4, _log_int(rng, 1, 256)))
        if kind == "prompt":
            batch, q_len = rng.randint(1, 3), _log_int(rng, 33, 2500)
            kv_len = q_len + _log_int(rng, 1, 8000)
        else:
            q_len = 1 if kind == "step" else rng.randint(2, 9)
            batch = _log_int(rng, 1, 128)
            kv_len = _log_int(rng, max(16, q_len), max(64, min(130000, 1000000 // batch)))
        c = _window("", dtype, batch, q_len, heads, kv_heads, head_dim, rng.choice((16, 32, 64, 128)),
                    kv_len, window, sinks, ragged=batch > 1 and rng.random() < 0.6)
    else:
        place = rng.choice(("step", "text", "text", "image", "video"))
        axes = {"image": 2, "video": 3}.get(place, 1)
        adjacent, factor = rng.random() < 0.3, rng.choice((1.0, 1.0, 1.1386, 0.9))
        base = rng.choice((1e4, 5e5, 1e6))
        values = _log_int(rng, 1 << 12, 1 << 26)
        if op == "rotate":
            head_dim = rng.choice((64, 72, 80, 96, 128, 128, 256))
            pairs = rng.choice((head_dim // 2, head_dim // 2, head_dim // 16 * 4))
            heads = rng.randint(1, 48)
            c = _rotate("", dtype, max(1, values // (heads * head_dim)), heads, head_dim,
                        _split_pairs(rng, pairs, axes), place, base, adjacent, factor, rng.random() < 0.4)
        else:
            head_dim = rng.choice((64, 80, 96, 112, 128, 128, 256))
            pairs = rng.choice((head_dim // 2, head_dim // 2, head_dim // 32 * 8))
            kv_heads = rng.randint(1, 12)
            heads = kv_heads * rng.choice((0, 1, 2, 4, 7))  # 0: no queries (a layer's cache filled apart)
            c = _append("", dtype, max(1, values // ((heads + kv_heads) * head_dim)), heads, kv_heads,
                        head_dim, rng.choice((16, 32, 64, 128)), _split_pairs(rng, pairs, axes), place,
                        base, adjacent, factor, rng.random() < 0.4)
    del c["name"]
    while work(c)["bytes"] > MOST_BYTES or work(c)["flops"] > MOST_FLOPS:
        for key in ("tokens", "batch", "q_len", "kv_len"):
            if c.get(key, 0) > 1:
                c[key] -= max(1, c[key] // 4)
        if op == "window":
            c["kv_len"] = max(c["kv_len"], c["q_len"])
    return c


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each sequence: a property of the
    case, not of the seed."""
    rng = random.Random("%(batch)d %(q_len)d %(kv_len)d" % case)
    B, nq, nk = case["batch"], case["q_len"], case["kv_len"]
    if not case["ragged"]:
        return [nq] * B, [nk] * B
    q, k = [], []
    for b in range(B):
        q.append(nq if b == 0 else rng.randint(1, nq))
        k.append(nk if b == 0 else max(q[-1], _log_int(rng, max(1, nk // 16), nk)))
    if B > 2:
        q[1], k[1] = (1, 0) if nq == 1 else (0, 0)  # an idle slot of the batch
    return q, k


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    hd = case["head_dim"]
    if case["op"] == "window":
        q, k = _lengths(case)
        w, s = case["window"], case["sinks"]
        pairs = tokens = 0
        for n, m in zip(q, k):
            for p in range(m - n, m):  # the positions of the new tokens
                if p >= 0:
                    pairs += min(w, p + 1) + min(s, max(0, p + 1 - w))
            if n and m:
                tokens += min(m, w + n - 1) + min(s, max(0, m - (w + n - 1)))
        row = 2 * case["kv_heads"] * hd
        return {"bytes": tokens * row * 9 / 16 + 2 * sum(q) * case["heads"] * hd * size,
                "flops": 4.0 * hd * case["heads"] * pairs}
    n, axes = case["tokens"], len(_sections(case))
    turned = 2 * sum(_sections(case))
    if case["op"] == "rotate":
        times = 2 if case["train"] else 1
        return {"bytes": times * n * 2 * case["heads"] * hd * size + n * 8 * axes,
                "flops": times * 3.0 * n * case["heads"] * turned}
    row = 2 * case["kv_heads"] * hd
    return {"bytes": n * (2 * row * size + 2 * row * 9 / 16 + 2 * case["heads"] * hd * size + 8 * (1 + axes)),
            "flops": n * (4.0 * row + 3.0 * (case["heads"] + case["kv_heads"]) * turned)}


# ------------------------------------------------------------- NVFP4 in plain fp32 torch
# A rounding decision compares |x| with a midpoint times s times S. The midpoint times s has at
# most 7 significant bits; with S split into halves of 12 bits both products are exact, so the
# fp32 comparison of (|x| - high) with low decides on exact values.

def _e4m3(dev):
    """E4M3 values of the bytes 0..255 as block scales: sign bit ignored, 0x7F (NaN) as zero."""
    b = torch.arange(256, device=dev) & 127
    e, m = b >> 3, (b & 7).float()
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.float() - 10), m * 2.0 ** -9)
    return v.masked_fill(b == 127, 0.0)


def _e2m1(dev):
    """Signed grid values of the codes 0..15."""
    c = torch.arange(16, device=dev)
    e, m = (c >> 1) & 3, (c & 1).float()
    return torch.where(e > 0, (1 + m / 2) * torch.exp2(e.float() - 1), m / 2) * (1 - 2.0 * (c >> 3))


def _plain_quantise(x, S):
    """Codes and block scale bytes of x [tokens, heads, head_dim] (fp32), S [heads]."""
    t, h, d = x.shape
    x = x.reshape(t, h, d // 16, 16)
    table = _e4m3(x.device)[:127]
    high = (S.view(torch.int32) & -4096).view(torch.float32)
    hi, lo = high.view(1, h, 1), (S - high).view(1, h, 1)
    amax = x.abs().amax(-1)
    mid = (table[1:] + table[:-1]) / 2                            # between bytes b and b + 1
    b = torch.bucketize(amax / (6 * S.view(1, h, 1)), mid)        # off by one at most
    for step in (0, 1):                                           # below, then above
        at = (b - 1 + step).clamp(0, 125)
        m6 = mid[at] * 6
        far, low = amax - m6 * hi, m6 * lo
        up = (far > low) | ((far == low) & (at % 2 == 1))
        b = torch.where(up, b, torch.minimum(b, at)) if step == 0 else torch.where(up, torch.maximum(b, at + 1), b)
    b = torch.where(amax > 0, b.clamp(1, 126), torch.zeros_like(b))
    s = table[b]
    ax, code = x.abs(), torch.zeros_like(x, dtype=torch.int64)
    hi, lo = hi.unsqueeze(-1), lo.unsqueeze(-1)
    for j in range(7):
        ts = s.unsqueeze(-1) * ((GRID[j] + GRID[j + 1]) / 2)
        far, low = ax - ts * hi, ts * lo
        code += (far >= low) if j % 2 else (far > low)
    code = torch.where(b.unsqueeze(-1) > 0, code, torch.zeros_like(code))
    code += 8 * ((x < 0) & (code > 0))
    return code.reshape(t, h, d), b


def _plain_values(code, byte, S):
    """fp32(G s S), S broadcast: one rounding, the product G s being exact."""
    g = _e2m1(code.device)[code.long()]
    s = _e4m3(code.device)[byte.long()].repeat_interleave(16, -1)
    return g * s * S


def _unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _plain_store(x, S, slots, codes, scales):
    ps = codes.shape[2]
    keep = (slots >= 0).nonzero().squeeze(1)
    c, b = _plain_quantise(x, S)
    c, b, slots = c[keep], b[keep], slots[keep]
    packed = (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)
    codes[slots // ps, :, slots % ps] = packed
    scales[slots // ps, :, slots % ps] = b.to(torch.uint8)


def _plain_load(codes, scales, S, slots, dtype):
    ps = codes.shape[2]
    at = slots.clamp(min=0)
    y = _plain_values(_unpack(codes[at // ps, :, at % ps]), scales[at // ps, :, at % ps], S.view(-1, 1))
    return torch.where((slots >= 0).view(-1, 1, 1), y, torch.zeros_like(y)).to(dtype)


# ------------------------------------------------------------------------- plain rotation

def _plain_table(st):
    """Cosines and sines [tokens, 1, pairs] in fp32, from angles in fp64."""
    angle = st["positions"].double()[st["axis"].long()].t() * st["inv_freq"]
    f = st["case"]["factor"]
    return (torch.cos(angle) * f).float().unsqueeze(1), (torch.sin(angle) * f).float().unsqueeze(1)


def _plain_rotate(x, table, adjacent):
    """fp32 rotation of x [tokens, heads, head_dim]; channels behind the pairs pass through."""
    c, s = table
    P = c.shape[-1]
    x = x.float()
    turn, rest = x[..., :2 * P], x[..., 2 * P:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if adjacent else (turn[..., :P], turn[..., P:])
    y, z = a * c - b * s, b * c + a * s
    pair = torch.stack((y, z), -1).flatten(-2) if adjacent else torch.cat((y, z), -1)
    return torch.cat((pair, rest), -1)


# -------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _positions(g, tokens, place):
    """Positions [axes, tokens] (int64). step: a new token of each of many sequences; text: packed
    prompts that start anywhere in a context; image: patch rows and columns; video: frames of
    patches, their corner where the text before them ends."""
    i = torch.arange(tokens, device=DEV)

    def some(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g, device=DEV)
    if place == "step":
        return some(0, 131072, tokens).view(1, -1)
    if place == "text":
        length = 4096
        return (some(0, 1000000, tokens // length + 1)[i // length] + i % length).view(1, -1)
    wide = int(some(20, 100, 1))
    if place == "image":
        return torch.stack((i // wide, i % wide))
    high = int(some(10, 60, 1))
    start = int(some(0, 30000, 1))
    return start + torch.stack((i // (wide * high), i // wide % high, i % wide))


def _frequencies(case):
    n = sum(_sections(case))
    w = case["base"] ** (-torch.arange(n, dtype=torch.float64) / n)
    axis = torch.cat([torch.full((m,), a, dtype=torch.int32) for a, m in enumerate(_sections(case))])
    return w.to(DEV), axis.to(DEV)


def _keys_values(g, tokens, heads, head_dim, dtype, spare=0):
    """Keys and values as slices of a fused projection's rows (``spare`` other heads first):
    normal, the keys with a few strong channels in every head. Also the other heads."""
    w = torch.randn(tokens, spare + 2 * heads, head_dim, generator=g, device=DEV)
    strong = 1 + 6 * (torch.rand(heads, head_dim, generator=g, device=DEV) < 0.03)
    w[:, spare:spare + heads] *= strong
    w = w.to(dtype)
    return w[:, spare:spare + heads], w[:, spare + heads:], w[:, :spare]


def _head_scales(x):
    return (x.float().abs().amax((0, 2)) / 2688).contiguous()


def _empty_cache(pages, case, g):
    """Cache memory as an allocator leaves it: any bytes."""
    ps, h, hd = case["page_size"], case["kv_heads"], case["head_dim"]

    def any_bytes(last):
        return torch.randint(0, 256, (pages, h, ps, last), generator=g, device=DEV, dtype=torch.uint8)
    return any_bytes(hd // 2), any_bytes(hd // 16), any_bytes(hd // 2), any_bytes(hd // 16)


def prepare(case, seed):
    g = _generator(seed)
    dtype, hd = DTYPES[case["dtype"]], case["head_dim"]
    st = {"op": case["op"], "dtype": dtype, "case": case}
    if case["op"] != "window":
        n = case["tokens"]
        st["inv_freq"], st["axis"] = _frequencies(case)
        st["positions"] = _positions(g, n, case["place"])
        if own:
            from scale_search_weights_amd import rotary
            st["rotary"] = rotary.Rotary(st["inv_freq"], st["axis"], axes=len(_sections(case)),
                                         adjacent=case["adjacent"], factor=case["factor"])
    if case["op"] == "rotate":
        # rows of a fused projection whose values follow (training: rows of their own)
        x = torch.randn(n, case["heads"] + (0 if case["train"] else 8), hd, generator=g, device=DEV).to(dtype)
        st["x"] = x[:, :case["heads"]]
        if case["train"]:
            st["x"].requires_grad_(own)
            st["grad"] = torch.randn(n, case["heads"], hd, generator=g, device=DEV).to(dtype)
        return st
    ps, h = case["page_size"], case["kv_heads"]
    if case["op"] == "append":
        pages = -(-n // ps) + 2
        order = torch.randperm(pages, generator=g, device=DEV)
        i = torch.arange(n, device=DEV)
        slots = order[i // ps] * ps + i % ps
        if case["skipped"]:  # the padding of a padded batch
            slots = torch.where(torch.rand(n, generator=g, device=DEV) < 0.1, torch.full_like(slots, -1), slots)
        st["k"], st["v"], st["q"] = _keys_values(g, n, h, hd, dtype, spare=case["heads"])
        st["S_k"], st["S_v"] = 1.5 * _head_scales(st["k"]), _head_scales(st["v"])  # a turned pair may grow
        st["cache"], st["slots"] = _empty_cache(pages, case, g), slots
    else:
        nq, nk = _lengths(case)
        per = [-(-m // ps) for m in nk]
        pages = sum(per) + 3
        order = torch.randperm(pages, generator=g, device=DEV)
        table = torch.zeros(case["batch"], max(1, -(-case["kv_len"] // ps)), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n]
            at += n
        st["table"] = table
        st["kv_lens"] = torch.tensor(nk, dtype=torch.int32, device=DEV)
        offs = [0]
        for n in nq:
            offs.append(offs[-1] + n)
        st["q_offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV)
        st["tokens"], st["max_q"], st["max_kv"] = offs[-1], max(nq), max(nk)
        st["uniform"] = min(nq) == max(nq)
        # every used page is filled a few thousand tokens at a time; the rest stays any bytes
        st["cache"] = _empty_cache(pages, case, g)
        used, step = at * ps, max(ps, (1 << 25) // (h * hd) // ps * ps)
        for lo in range(0, used, step):
            i = torch.arange(lo, min(used, lo + step), device=DEV)
            slots = order[i // ps] * ps + i % ps
            k, v, _ = _keys_values(g, i.numel(), h, hd, dtype)
            if lo == 0:
                st["S_k"], st["S_v"] = _head_scales(k), _head_scales(v)
            _plain_store(k.float(), st["S_k"], slots, *st["cache"][:2])
            _plain_store(v.float(), st["S_v"], slots, *st["cache"][2:])
        qkv = torch.randn(offs[-1], case["heads"] + 2 * h, hd, generator=g, device=DEV).to(dtype)
        st["q"] = qkv[:, :case["heads"]]
        st["scale"] = hd ** -0.5
    if own:
        from scale_search_weights_amd import kvcache
        st["handle"] = kvcache.KVCache(*st["cache"], st["S_k"], st["S_v"])
    return st


# ------------------------------------------------------------------------- plain attention

def _plain_window(st):
    """The tokens that some new query of a sequence sees, gathered: its first ones and the
    windows' union. Scores of what a query does not see are -inf."""
    c, q = st["case"], st["q"]
    kc, ks, vc, vs = st["cache"]
    B, n, H, h, hd = c["batch"], st["max_q"], c["heads"], c["kv_heads"], c["head_dim"]
    w, first, ps = c["window"], c["sinks"], c["page_size"]
    lens = st["kv_lens"].long().view(B, 1)
    start = st["q_offsets"].long()
    count = (start[1:] - start[:-1]).view(B, 1)
    i = torch.arange(n, device=q.device).view(1, n)
    at = (start[:-1].view(B, 1) + i).clamp(max=max(0, st["tokens"] - 1))
    qp = q.float()[at].view(B, n, h, H // h, hd).permute(0, 2, 3, 1, 4).reshape(B, h, -1, hd) * st["scale"]
    L = min(st["max_kv"], first + w + n - 1)
    u = torch.arange(L, device=q.device).view(1, L)
    # gathered token u: itself among the first, else counted from the first row's window
    t = torch.where(u < first, u, u + (lens - count - w + 1 - first).clamp(min=0))
    stands = (lens - count + i).view(B, n, 1)
    t3 = t.view(B, 1, L)
    seen = (t3 <= stands) & ((t3 > stands - w) | (t3 < first)) & (t3 < lens.view(B, 1, 1))
    t = torch.minimum(t, (lens - 1).clamp(min=0))
    page, offset = torch.gather(st["table"].long(), 1, t // ps), t % ps

    def rows(codes, scales, S):
        x = _plain_values(_unpack(codes[page, :, offset]), scales[page, :, offset], S.view(-1, 1))
        return x.transpose(1, 2).contiguous()  # [batch, heads, tokens, head_dim]
    k = rows(kc, ks, st["S_k"])
    s = torch.matmul(qp, k.transpose(-1, -2)).view(B, h, H // h, n, L)
    del k
    s = s.masked_fill(~seen.view(B, 1, 1, n, L), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s = torch.exp(s.sub_(m))
    z = s.sum(-1, keepdim=True)
    z = torch.where(z == 0, torch.ones_like(z), z)
    o = torch.matmul(s.view(B, h, -1, L), rows(vc, vs, st["S_v"]))
    o = (o.view(B, h, H // h, n, hd) / z).permute(0, 3, 1, 2, 4).reshape(B, n, H, hd)
    tok = torch.arange(st["tokens"], device=q.device)
    b = torch.bucketize(tok, start[1:], right=True)
    return o[b, tok - start[b]].to(st["dtype"])


def run(state):
    st, c = state, state["case"]
    if own:
        from scale_search_weights_amd import kvcache, rotary
        if st["op"] == "rotate":
            y = rotary.rotate(st["x"], st["positions"], st["rotary"])
            if not c["train"]:
                return y
            return y.detach(), torch.autograd.grad(y, st["x"], st["grad"])[0]
        if st["op"] == "append":
            q = kvcache.append(st["handle"], st["k"], st["v"], st["slots"], st["positions"], st["rotary"],
                               q=st["q"] if c["heads"] else None)
            k, v = kvcache.read(st["handle"], st["slots"], st["dtype"])
            return (q, k, v) if c["heads"] else (k, v)
        return kvcache.attention(
            st["handle"], st["q"], st["table"], st["kv_lens"],
            q_offsets=None if st["uniform"] else st["q_offsets"], max_q=st["max_q"],
            max_kv=st["max_kv"], scale=st["scale"], window=c["window"], sinks=c["sinks"])
    if st["op"] == "window":
        return _plain_window(st)
    cos, sin = _plain_table(st)
    if st["op"] == "rotate":
        y = _plain_rotate(st["x"], (cos, sin), c["adjacent"]).to(st["dtype"])
        if not c["train"]:
            return y
        return y, _plain_rotate(st["grad"], (cos, -sin), c["adjacent"]).to(st["dtype"])
    kc, ks, vc, vs = st["cache"]
    _plain_store(_plain_rotate(st["k"], (cos, sin), c["adjacent"]), st["S_k"], st["slots"], kc, ks)
    _plain_store(st["v"].float(), st["S_v"], st["slots"], vc, vs)
    k = _plain_load(kc, ks, st["S_k"], st["slots"], st["dtype"])
    v = _plain_load(vc, vs, st["S_v"], st["slots"], st["dtype"])
    if not c["heads"]:
        return k, v
    return _plain_rotate(st["q"], (cos, sin), c["adjacent"]).to(st["dtype"]), k, v


# --------------------------------------------------------------------------- 64-bit values

def _nearest(a, values, unit):
    """Index of the value nearest to a / unit, ties to the even index, per element: distances
    |a - value unit| in 64 bits, over all values."""
    best = torch.full_like(a, math.inf)
    index = torch.zeros(a.shape, dtype=torch.int64, device=a.device)
    for n, v in enumerate(values):
        d = (a - v * unit).abs()
        take = (d < best) | ((d == best) & (n % 2 == 0))
        index = torch.where(take, n, index)
        best = torch.where(take, d, best)
    return index


def _exact_round(x, S):
    t, h, d = x.shape
    x = x.double().reshape(t, h, d // 16, 16)
    S = S.double().view(1, h, 1)
    e4m3 = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]
    amax = x.abs().amax(-1)
    byte = _nearest(amax, e4m3, 6 * S)
    byte = torch.where(amax > 0, byte.clamp(min=1), 0)
    unit = (torch.tensor(e4m3, dtype=torch.float64, device=x.device)[byte] * S).unsqueeze(-1)
    k = _nearest(x.abs(), GRID, unit)
    return (torch.tensor(GRID, dtype=torch.float64, device=x.device)[k] * unit * x.sign()).view(t, h, d)


def _exact_turn(x, st, sign=1.0):
    """Each pair as a complex number times factor e^(i angle), in 64 bits, by head to bound memory."""
    c = st["case"]
    P = st["inv_freq"].numel()
    angle = torch.stack([st["positions"][int(a)].double() * w for a, w in
                         zip(st["axis"].tolist(), st["inv_freq"].tolist())], -1)
    turn = torch.polar(torch.full_like(angle, c["factor"]), sign * angle)
    y = x.detach().double().clone()
    for head in range(x.shape[1]):
        r = y[:, head]
        if c["adjacent"]:
            z = torch.view_as_complex(r[:, :2 * P].reshape(-1, P, 2).contiguous()) * turn
            y[:, head, :2 * P] = torch.view_as_real(z).reshape(-1, 2 * P)
        else:
            z = torch.complex(r[:, :P].contiguous(), r[:, P:2 * P].contiguous()) * turn
            y[:, head, :P], y[:, head, P:2 * P] = z.real, z.imag
    return y


def _exact_cached(codes, scales, S, page, offset):
    """Values at (page, offset) of every head: [..., heads, head_dim] in 64 bits."""
    c = codes[page, :, offset].long()
    lo, hi = c % 16, c // 16
    c = torch.stack((lo, hi), -1).flatten(-2)
    e = scales[page, :, offset].long()
    mant, exp = e % 8, e // 8 % 16
    s = torch.where(exp > 0, (8.0 + mant) * 2.0 ** (exp.double() - 10), mant.double() / 512)
    mag = torch.tensor(GRID, dtype=torch.float64, device=c.device)[c % 8]
    return mag * torch.where(c >= 8, -1.0, 1.0).double() * s.repeat_interleave(16, -1) * S.double().unsqueeze(-1)


def exact(case, seed):
    global own
    before, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = before
    if case["op"] == "rotate":
        y = _exact_turn(st["x"], st)
        return (y, _exact_turn(st["grad"], st, -1.0)) if case["train"] else y
    if case["op"] == "append":
        seen = (st["slots"] >= 0).double().view(-1, 1, 1)
        parts = []
        for x, S in ((_exact_turn(st["k"], st), st["S_k"]), (st["v"], st["S_v"])):
            step = 1 + (1 << 25) // (x.shape[1] * x.shape[2])
            parts.append(torch.cat([_exact_round(p, S) for p in x.split(step)]) * seen)
        return (_exact_turn(st["q"], st), *parts) if case["heads"] else tuple(parts)
    ps = case["page_size"]
    kc, ks, vc, vs = st["cache"]
    q, H, h = st["q"].double(), case["heads"], case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    starts, lens = st["q_offsets"].tolist(), st["kv_lens"].tolist()
    for b in range(case["batch"]):
        lo, hi, m = starts[b], starts[b + 1], lens[b]
        n = hi - lo
        if n == 0 or m == 0:
            continue
        near = max(0, m - n - case["window"] + 1)  # no row's window begins before
        t = torch.arange(m, device=q.device)
        t = t[(t < case["sinks"]) | (t >= near)]
        page = st["table"][b].long()[t // ps]
        k = _exact_cached(kc, ks, st["S_k"], page, t % ps).transpose(0, 1).contiguous()
        v = _exact_cached(vc, vs, st["S_v"], page, t % ps).transpose(0, 1).contiguous()
        p = torch.arange(m - n, m, device=q.device).view(-1, 1)
        hidden = (t > p) | ((t <= p - case["window"]) & (t >= case["sinks"]))
        for head in range(H):
            s = q[lo:hi, head] @ k[head // (H // h)].T * st["scale"]
            s = s.masked_fill(hidden, -math.inf)
            out[lo:hi, head] = torch.nan_to_num(torch.softmax(s, -1)) @ v[head // (H // h)]
    return out
