"""Decoding with keys and values cached in NVFP4.

One attention layer with random projections serves a batch of users behind one long shared prompt:

1. the tensor scale of each key/value head comes from a calibration pass over the prompt's keys
   and values (amax / 2688, with some room for values the prompt does not show);
2. the prompt's keys and values are quantised into pages as they are written, and the prompt's own
   outputs are computed from the cache (causal attention of many queries);
3. every decoding step writes one new token of every user and attends over the shared prompt and
   the user's own tokens (one query each);
4. at the end the cache is read back, and the last outputs are compared with attention over the
   keys and values before quantisation.

    python examples/kv_decode.py [--users 64] [--prompt 8192] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from scale_search_weights_amd import kvcache, nvfp4  # noqa: E402

HEADS, KV_HEADS, HEAD_DIM, HIDDEN, PAGE = 32, 8, 128, 4096, 64


def run(users: int = 64, prompt: int = 8192, steps: int = 32, seed: int = 0, device: str = "cuda") -> dict:
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=device) * scale).to(torch.bfloat16)

    w = normal(HIDDEN, (HEADS + 2 * KV_HEADS) * HEAD_DIM, scale=HIDDEN ** -0.5)

    def project(x):  # queries, keys and values as slices of one product's rows
        y = (x @ w).view(-1, HEADS + 2 * KV_HEADS, HEAD_DIM)
        return y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]

    # 1. head scales
    q, k, v = project(normal(prompt, HIDDEN))
    room = 1.25
    S_k = nvfp4.global_scale(k.transpose(0, 1).contiguous()) * room
    S_v = nvfp4.global_scale(v.transpose(0, 1).contiguous()) * room

    # 2. the prompt, in the first pages; the users' pages follow, enough for their steps
    prefix = -(-prompt // PAGE)
    own = -(-steps // PAGE)
    cache = kvcache.KVCache.empty(prefix + users * own, PAGE, KV_HEADS, HEAD_DIM, S_k, S_v)
    prefix_pages = torch.arange(prefix, dtype=torch.int32, device=device)
    table = prefix + torch.arange(users * own, dtype=torch.int32, device=device).view(users, own)
    kvcache.write(cache, k, v, torch.arange(prompt, device=device))
    lens = torch.tensor([prompt], dtype=torch.int32, device=device)
    prompt_out = kvcache.attention(cache, q, prefix_pages.view(1, -1), lens, max_kv=prompt)

    # 3. decoding steps
    keys, values = [], []
    lens = torch.zeros(users, dtype=torch.int32, device=device)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for step in range(steps):
        q1, k1, v1 = project(normal(users, HIDDEN))
        slots = table[:, step // PAGE].long() * PAGE + step % PAGE
        kvcache.write(cache, k1, v1, slots)
        lens += 1
        out = kvcache.attention(cache, q1, table, lens, max_kv=step + 1, prefix_pages=prefix_pages,
                                prefix_len=prompt)
        keys.append(k1), values.append(v1)
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start

    # 4. what the cache stands for, and the last step without quantisation
    read_k, _ = kvcache.read(cache, torch.arange(prompt, device=device))
    own_k, own_v = (torch.stack(t).float() for t in (keys, values))  # [steps, users, heads, dim]
    group, worst = HEADS // KV_HEADS, 0.0
    for user in range(min(users, 4)):
        kk = torch.cat((k.float(), own_k[:, user]))
        vv = torch.cat((v.float(), own_v[:, user]))
        qq = q1[user].float().view(KV_HEADS, group, HEAD_DIM)
        s = torch.matmul(qq, kk.permute(1, 2, 0).contiguous()) * HEAD_DIM ** -0.5
        want = torch.matmul(torch.softmax(s, -1), vv.transpose(0, 1).contiguous()).view(HEADS, HEAD_DIM)
        worst = max(worst, float((out[user].float() - want).norm() / want.norm()))
    cached = prefix * PAGE * KV_HEADS * HEAD_DIM
    return {"ms_per_step": 1e3 * seconds / steps, "output_error": worst,
            "key_error": float((read_k.float() - k.float()).norm() / k.float().norm()),
            "bytes_per_value": (cache.k_codes[:prefix].numel() + cache.k_scales[:prefix].numel()) / cached,
            "prompt_out": prompt_out, "out": out}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    r = run(a.users, a.prompt, a.steps)
    print(f"{a.users} users behind a prompt of {a.prompt} tokens, {a.steps} steps: {r['ms_per_step']:.3f} ms a step; "
          f"{r['bytes_per_value']} bytes a cached value; keys off by {r['key_error']:.3f} (relative norm), "
          f"the last outputs by {r['output_error']:.3f} against unquantised attention")


if __name__ == "__main__":
    main()
