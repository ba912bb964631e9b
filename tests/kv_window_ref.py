"""Plain 64-bit reference of attention over a window and sinks (CPU, torch double), from its definition;
inputs are kvcache_ref.make's, bounds those of test_gpu_kvcache.py with fp16's smallest step."""
import math

import torch

import kvcache_ref as ref


def seen(n, m, window, sinks):
    """[n, m]: which tokens the last n of m positions see."""
    P = m - n + torch.arange(n).view(-1, 1)
    t = torch.arange(m).view(1, -1)
    return (t <= P) & ((t > P - window) | (t < sinks))


def attention(c, window, sinks, scale):
    """out, lse, A = sum_t p_t |v_t|, B = max_t |scale| sum_d |q_d k_td|, V = sum_t |v_t| over what a row
    sees; tokens of pages outside the cache are hidden."""
    kc, ks, vc, vs, S_k, S_v, ps = c["cache"]
    q, offs = c["q"], c["q_offsets"]
    T, H, hd = q.shape
    G = H // kc.shape[1]
    out, A, V = (torch.zeros(T, H, hd, dtype=torch.float64) for _ in range(3))
    lse, B = torch.full((T, H), -math.inf, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for b in range(len(offs) - 1):
        lo, hi, m = int(offs[b]), int(offs[b + 1]), int(c["kv_lens"][b])
        if hi == lo or m <= 0:
            continue
        mask = seen(hi - lo, m, window, sinks)
        t = mask.any(0).nonzero().squeeze(1)  # pages of tokens that no row sees may not exist
        page = c["table"][b].long()[t // ps]
        ok = (page >= 0) & (page < kc.shape[0])
        t, page = t[ok], page[ok]
        k = ref.values(kc[page, :, t % ps], ks[page, :, t % ps], S_k.view(1, -1, 1)).transpose(0, 1)
        v = ref.values(vc[page, :, t % ps], vs[page, :, t % ps], S_v.view(1, -1, 1)).transpose(0, 1)
        mask = mask[:, t]
        for h in range(H):
            qq, kk, vv = q[lo:hi, h].double(), k[h // G], v[h // G]
            s = (qq @ kk.T * scale).masked_fill(~mask, -math.inf)
            B[lo:hi, h] = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(~mask, 0).amax(1) if t.numel() else 0
            lse[lo:hi, h] = torch.logsumexp(s, 1)
            p = torch.nan_to_num(torch.softmax(s, 1))
            out[lo:hi, h], A[lo:hi, h], V[lo:hi, h] = p @ vv, p @ vv.abs(), mask.double() @ vv.abs()
    return out, lse, A, B, V


def check(c, got, window, sinks, scale=None):
    out, lse = (t.cpu() for t in got)
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    o, z, A, B, V = attention(c, window, sinks, scale)
    bf = out.dtype == torch.bfloat16
    d = 2 * 1.05 * 2.0 ** -19 * B.unsqueeze(-1) + (2.0 ** -11 if bf else 2.0 ** -21) + 2.0 ** -20
    tol = A * d + o.abs() * (2.0 ** -8 if bf else 2.0 ** -22) + V * (2.0 ** -32 if bf else 2.0 ** -38)
    err = (out.double() - o).abs()
    assert torch.isfinite(out.float()).all()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0, (worst, err.max().item(), (err > tol).nonzero()[:5].tolist())
    empty = torch.isneginf(z)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    dl = ((lse.double() - z).abs() - (2.0 ** -19 * B + 2.0 ** -19 + 2.0 ** -22 * z.abs()))[~empty]
    assert not dl.numel() or dl.max() <= 0, dl.max()
