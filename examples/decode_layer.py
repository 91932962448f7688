"""A decoder layer's attention half on this framework: W12 products around a paged
key-value cache.

    python examples/decode_layer.py [--cache q8] [--steps 64] [--draft 4]

Per step: q, k and v in one grouped W12 launch; the page plan (once for all layers
of a model); norm, rotation and the cache write; attention; the output product.
With --draft n every step brings n + 1 tokens of each request (a verification of n
drafted ones), of which a random number is accepted: the others' pages and slots are
simply planned again.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_bit_weight_encode_gb300 import KVCache, KVPages, W12Group, W12Weight, w12  # noqa: E402

MAX_TOKENS = 32  # of a W12 product


def rope_table(rows, rot, base=1e6, device="cuda"):
    freq = base ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    angle = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class AttentionBlock:
    """x [tokens, hidden] -> x + o(attention(q, k, v)), with its own layer's cache.
    Weights are BF16 device tensors (wq, wk, wv, wo) and are encoded to W12 here."""

    def __init__(self, wq, wk, wv, wo, q_norm, k_norm, head_dim, pages, num_pages, cache="bf16"):
        self.qkv = W12Group([W12Weight.from_device(w) for w in (wq, wk, wv)])
        self.o = W12Weight.from_device(wo)
        self.q_norm, self.k_norm = q_norm, k_norm
        self.cache = KVCache.empty(num_pages, pages.page_size, wk.shape[0] // head_dim, head_dim, cache)

    def __call__(self, x, step, rope):
        # a W12 product takes up to 32 tokens
        parts = [self.qkv.gemm(part) for part in x.split(MAX_TOKENS)]
        q, k, v = (torch.cat(t) for t in zip(*parts))
        q = self.cache.store(q, k, v, step, q_norm=self.q_norm, k_norm=self.k_norm, rope=rope)
        y = self.cache.attend(q, step).view(x.shape[0], -1)
        return x + torch.cat([self.o.gemm(part) for part in y.split(MAX_TOKENS)])


def make_block(hidden, heads, kv_heads, head_dim, pages, num_pages, cache="bf16", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: (torch.randn(*s, device="cuda", generator=g) * s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
    weights = (rnd(heads * head_dim, hidden), rnd(kv_heads * head_dim, hidden), rnd(kv_heads * head_dim, hidden),
               rnd(hidden, heads * head_dim))
    norms = tuple((1 + 0.1 * torch.randn(head_dim, device="cuda", generator=g)).to(torch.bfloat16) for _ in range(2))
    return AttentionBlock(*weights, *norms, head_dim, pages, num_pages, cache), weights, norms


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=("bf16", "q8"), default="bf16")
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--draft", type=int, default=3)
    ap.add_argument("--page", type=int, default=16)
    a = ap.parse_args()
    hidden, heads, kv_heads, head_dim = 5120, 48, 8, 128  # the benchmark's decoder layer
    per, most = a.draft + 1, (a.steps + 1) * (a.draft + 1)
    blocks = -(-most // a.page)
    num_pages = a.requests * blocks
    pages = KVPages.create(num_pages, a.page, a.requests, blocks)
    block, _, _ = make_block(hidden, heads, kv_heads, head_dim, pages, num_pages, a.cache)
    rope = rope_table(most, head_dim)
    step = pages.step(a.requests * per, max_new=per)
    lens = torch.zeros(a.requests, dtype=torch.int32, device="cuda")
    new = torch.full_like(lens, per)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(a.steps):
        x = torch.randn(a.requests * per, hidden, device="cuda", generator=g).to(torch.bfloat16)
        pages.plan(lens, new, step)
        y = block(x, step, rope)
        accepted = torch.randint(1, per + 1, (a.requests,), device="cuda", generator=g, dtype=torch.int32)
        lens += accepted  # the rejected tokens' slots are written again in the next step
    w12.w12_check_status()
    # the finished requests' pages go back
    pages.plan(torch.zeros_like(lens), torch.zeros_like(new), pages.step(0), trim=True)
    w12.w12_check_status()
    head, tail = pages.ring_state.tolist()
    print(f"{a.steps} steps of {a.requests} requests x {per} tokens, {a.cache} cache: cached lengths {lens.tolist()}, "
          f"last output {tuple(y.shape)} rms {float(y.float().square().mean().sqrt()):.3f}, "
          f"{tail - head} of {num_pages} pages free again")


if __name__ == "__main__":
    main()
