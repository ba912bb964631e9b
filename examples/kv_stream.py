"""Streaming in bounded memory: rotary positions, keys and values cached in NVFP4, a sliding window with sinks.

One attention layer with random projections serves a few users for longer than their pages last:

1. a prompt of text, a video and text again gets positions on three axes (time, height, width);
2. the prompt goes in by chunks: `append` turns a chunk's keys and queries and quantises keys and values
   into their pages in one launch, then its queries attend over the window and the first tokens;
3. decoding goes on in the same way, a token a step. A user owns the pages of the first tokens and a ring of
   pages for the window; whatever falls out of the window is overwritten;
4. at the end the last outputs are compared with attention over the turned keys and the values before
   quantisation.

    python examples/kv_stream.py [--users 8] [--steps 200] [--window 512]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from scale_search_weights_amd import kvcache, rotary  # noqa: E402

HEADS, KV_HEADS, HEAD_DIM, HIDDEN, PAGE, SINKS, CHUNK = 16, 4, 128, 2048, 64, 4, 256


def prompt_positions(before: int, frames: int, high: int, wide: int, after: int) -> torch.Tensor:
    """[3, tokens]: text counts all axes up together, a video's patches by frame, row and column from
    where the text stopped, and text goes on behind the largest of them."""
    i = torch.arange(frames * high * wide)
    video = before + torch.stack((i // (high * wide), i // wide % high, i % wide))
    text = torch.arange(before).expand(3, -1)
    more = int(video.max()) + 1 + torch.arange(after).expand(3, -1)
    return torch.cat((text, video, more), 1)


def run(users: int = 8, steps: int = 200, window: int = 512, seed: int = 0, device: str = "cuda") -> dict:
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=device) * scale).to(torch.bfloat16)

    w = normal(HIDDEN, (HEADS + 2 * KV_HEADS) * HEAD_DIM, scale=HIDDEN ** -0.5)
    rot = rotary.Rotary.create(HEAD_DIM, base=1e6, sections=(16, 24, 24), device=device)

    def project(x):  # queries, keys and values as slices of one product's rows
        y = (x @ w).view(-1, HEADS + 2 * KV_HEADS, HEAD_DIM)
        return y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]

    # 1. one prompt's positions; every user has its own tokens
    pos = prompt_positions(100, 10, 9, 16, 300).to(device)
    prompt = pos.shape[1]
    total = prompt + steps

    # pages: those of the sinks, then a ring that holds the window and a chunk
    first, ring = -(-SINKS // PAGE), -(-(window + CHUNK) // PAGE) + 1
    page = torch.arange(-(-total // PAGE), device=device)
    page = torch.where(page < first, page, first + (page - first) % ring)
    table = (page + (first + ring) * torch.arange(users, device=device).view(-1, 1)).int()
    S = torch.full((KV_HEADS,), 6.0 / 2688, device=device)  # what normal projections stay under
    cache = kvcache.KVCache.empty(users * (first + ring), PAGE, KV_HEADS, HEAD_DIM, S, S)

    def slots(lo, hi):  # of tokens lo .. hi - 1 of every user
        t = torch.arange(lo, hi, device=device)
        return (table[:, t // PAGE].long() * PAGE + t % PAGE).reshape(-1)

    keys, values, out = [], [], None

    def step(lo, hi, positions):  # positions [3, hi - lo], the same for every user
        nonlocal out
        q, k, v = project(normal(users * (hi - lo), HIDDEN))
        p = positions.repeat(1, users)
        keys.append(rotary.rotate(k.float(), p, rot).view(users, hi - lo, KV_HEADS, HEAD_DIM))  # for the comparison
        values.append(v.float().view(users, hi - lo, KV_HEADS, HEAD_DIM))
        q = kvcache.append(cache, k, v, slots(lo, hi), p, rot, q=q)
        lens = torch.full((users,), hi, dtype=torch.int32, device=device)
        out = kvcache.attention(cache, q, table, lens, max_kv=hi, window=window, sinks=SINKS)
        return q

    # 2. the prompt by chunks
    for lo in range(0, prompt, CHUNK):
        hi = min(prompt, lo + CHUNK)
        q = step(lo, hi, pos[:, lo:hi])

    # 3. decoding: text positions that go on
    torch.cuda.synchronize()
    start = time.perf_counter()
    for n in range(steps):
        q = step(prompt + n, prompt + n + 1, pos[:, -1:] + 1 + n)
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start

    # 4. the last step without quantisation
    t = torch.arange(total, device=device)
    seen = (t < SINKS) | (t > total - 1 - window)
    group, worst = HEADS // KV_HEADS, 0.0
    for user in range(min(users, 4)):
        kk, vv = (torch.cat([x[user] for x in xs])[seen] for xs in (keys, values))
        qq = q[user].float().view(KV_HEADS, group, HEAD_DIM)
        s = torch.matmul(qq, kk.permute(1, 2, 0).contiguous()) * HEAD_DIM ** -0.5
        want = torch.matmul(torch.softmax(s, -1), vv.transpose(0, 1).contiguous()).view(HEADS, HEAD_DIM)
        worst = max(worst, float((out[user].float() - want).norm() / want.norm()))
    return {"ms_per_step": 1e3 * seconds / max(1, steps), "output_error": worst, "tokens": total,
            "held": (first + ring) * PAGE, "out": out}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--users", type=int, default=8)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--window", type=int, default=512)
    a = ap.parse_args()
    r = run(a.users, a.steps, a.window)
    print(f"{a.users} users, {r['tokens']} tokens each in pages for {r['held']}, window {a.window}: {r['ms_per_step']:.3f} ms "
          f"a step; the last outputs are off by {r['output_error']:.3f} against unquantised attention")


if __name__ == "__main__":
    main()
