"""Plain 64-bit reference of the NVFP4 key/value cache (CPU, torch double), written from the
format's definition, and a seeded case builder shared by the tests."""
import math

import numpy as np
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3(byte):
    """Block scale of a byte: E4M3 magnitude, 0x7F as zero."""
    b = byte.long() & 127
    e, m = b >> 3, (b & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m / 512)
    return torch.where(b == 127, torch.zeros_like(v), v)


def values(codes, scales, S):
    """Exact G s S of packed codes [..., heads, *, hd/2]; S broadcast against [..., 1]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = GRID[c & 7] * torch.where(c > 7, -1.0, 1.0).double()
    return v * e4m3(scales).repeat_interleave(16, -1) * S.double()


def token_rows(codes, scales, S, pages, n, page_size):
    """[heads, n, hd] of the first n tokens of a page list; tokens of pages outside the cache
    come out as NaN (they are hidden)."""
    t = torch.arange(n)
    page = pages.long()[t // page_size] if n else t
    ok = (page >= 0) & (page < codes.shape[0])
    at = page.clamp(0, max(0, codes.shape[0] - 1))
    v = values(codes[at, :, t % page_size], scales[at, :, t % page_size], S.view(1, -1, 1))
    v[~ok] = math.nan
    return v.transpose(0, 1)


def attention(cache, q, table, kv_lens, q_offsets, prefix_pages, prefix_len, scale, causal):
    """out, lse, and per row the bounds' scales: A = sum_t p_t |v_t| and V = sum_t |v_t| over the
    seen tokens (per channel), and B = max_t |scale| sum_d |q_d k_td|."""
    kc, ks, vc, vs, S_k, S_v, ps = cache
    T, H, hd = q.shape
    G = H // kc.shape[1]
    out, A = torch.zeros(T, H, hd, dtype=torch.float64), torch.zeros(T, H, hd, dtype=torch.float64)
    V = torch.zeros(T, H, hd, dtype=torch.float64)
    lse, B = torch.full((T, H), -math.inf, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for b in range(len(q_offsets) - 1):
        lo, hi = int(q_offsets[b]), int(q_offsets[b + 1])
        n, m = hi - lo, int(kv_lens[b]) if kv_lens is not None else 0
        parts_k, parts_v = [], []
        if prefix_len:
            parts_k.append(token_rows(kc, ks, S_k, prefix_pages, prefix_len, ps))
            parts_v.append(token_rows(vc, vs, S_v, prefix_pages, prefix_len, ps))
        if m:
            parts_k.append(token_rows(kc, ks, S_k, table[b], m, ps))
            parts_v.append(token_rows(vc, vs, S_v, table[b], m, ps))
        if not parts_k or not n:
            continue
        k, v = torch.cat(parts_k, 1), torch.cat(parts_v, 1)
        P = k.shape[1] - m
        i, j = torch.arange(n).view(-1, 1), torch.arange(P + m).view(1, -1)
        for h in range(H):
            kk, vv = k[h // G], v[h // G]
            hidden = torch.isnan(kk[:, 0]).view(1, -1).expand(n, -1).clone()
            if causal:
                hidden |= (j >= P) & (j - P > m - n + i)
            kk, vv = torch.nan_to_num(kk), torch.nan_to_num(vv)
            qq = q[lo:hi, h].double()
            s = (qq @ kk.T * scale).masked_fill(hidden, -math.inf)
            B[lo:hi, h] = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(hidden, 0).amax(1)
            lse[lo:hi, h] = torch.logsumexp(s, 1)
            p = torch.nan_to_num(torch.softmax(s, 1))
            out[lo:hi, h], A[lo:hi, h] = p @ vv, p @ vv.abs()
            V[lo:hi, h] = (~hidden).double() @ vv.abs()
    return out, lse, A, B, V


def any_bytes(rng, shape):
    """Cache memory as found: any bytes, NaN scales among them."""
    x = rng.integers(0, 256, shape, dtype=np.uint8)
    x[rng.random(shape) < 0.2] = 0x7F
    return torch.from_numpy(x)


def make(seed, dtype, q_lens, kv_lens, heads, kv_heads, hd, page_size, prefix=0, spare_pages=2,
         q_scale=1.0):
    """Pages in random order holding random codes and finite block scales for every token in
    use, any bytes elsewhere; queries as a slice of wider rows."""
    rng = np.random.default_rng(seed)
    per = [-(-m // page_size) for m in kv_lens]
    np_ = -(-prefix // page_size)
    pages = sum(per) + np_ + spare_pages
    shape = (pages, kv_heads, page_size)
    kc, vc = any_bytes(rng, shape + (hd // 2,)), any_bytes(rng, shape + (hd // 2,))
    ks, vs = any_bytes(rng, shape + (hd // 16,)), any_bytes(rng, shape + (hd // 16,))
    order = rng.permutation(pages)
    prefix_pages = torch.from_numpy(order[:np_].astype(np.int32))
    table = torch.from_numpy(rng.integers(0, pages, (len(kv_lens), max([1] + per) + 1)).astype(np.int32))
    at = np_
    for b, n in enumerate(per):
        table[b, :n] = torch.from_numpy(order[at:at + n].astype(np.int32))
        at += n

    def fill(page_list, n):
        t = np.arange(n)
        for s in (ks, vs):
            # block scales within a factor of four of 448/12, a few zeros and subnormals
            good = rng.integers(0x58, 0x68, (n, kv_heads, hd // 16)).astype(np.uint8)
            good[rng.random(good.shape) < 0.02] = 0
            good[rng.random(good.shape) < 0.02] = 3
            s[page_list[t // page_size], :, t % page_size] = torch.from_numpy(good)
    fill(prefix_pages.numpy(), prefix)
    for b, m in enumerate(kv_lens):
        fill(table[b].numpy(), m)
    S_k = torch.from_numpy((rng.random(kv_heads) * 0.01 + 0.004).astype(np.float32))
    S_v = torch.from_numpy((rng.random(kv_heads) * 0.02 + 0.003).astype(np.float32))
    offs = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    wide = torch.from_numpy(rng.standard_normal((int(offs[-1]), heads + 2, hd + 8 * (hd % 32 == 0))).astype(np.float32))
    q = (wide * q_scale).to(dtype)[:, 1:1 + heads, :hd]
    return dict(cache=(kc, ks, vc, vs, S_k, S_v, page_size), q=q, table=table,
                kv_lens=torch.tensor(kv_lens, dtype=torch.int32), q_offsets=torch.from_numpy(offs),
                prefix_pages=prefix_pages, prefix_len=prefix, max_q=max([0] + list(q_lens)),
                max_kv=max([0] + list(kv_lens)))
