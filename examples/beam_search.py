"""Beam search on this framework: W12 layers around paged caches whose pages the beams share.

    python examples/beam_search.py [--beams 4] [--cache q8] [--steps 24]

A prompt is cached once, in the pages of its request's first beam.  Then, per step: the
best continuations of all beams (Beams.select); page tables that go on from their parents'
(KVPages.fork: full pages are shared, a partly filled one goes to one beam and is copied for
the others); those copies in every layer's cache; and a decoding step in which the keys
that a request's beams have in common are read once for all of them.  From the second
step on this is one CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "examples")):
    if path not in sys.path:
        sys.path.insert(0, path)

from decode_layer import MAX_TOKENS, make_block, rope_table  # noqa: E402

from lossless_bit_weight_encode_gb300 import Beams, KVCopies, KVPages, KVPrefix, W12Weight, w12  # noqa: E402


class BeamSearch:
    """``layers`` random attention blocks between an embedding and an LM head over ``vocab``
    tokens, searched with ``beams`` beams for each of ``requests`` prompts."""

    def __init__(self, requests, beams, vocab=4001, layers=2, hidden=512, heads=12, kv_heads=2, head_dim=64,
                 page=16, max_len=256, eos=0, cache="bf16", seed=0):
        self.requests, self.beams, self.rows = requests, beams, requests * beams
        blocks = -(-max_len // page)
        self.pages = KVPages.create(self.rows * blocks, page, self.rows, blocks, shared=True)
        make = lambda i: make_block(hidden, heads, kv_heads, head_dim, self.pages, self.rows * blocks, cache,  # noqa: E731
                                    seed + i)[0]
        self.blocks = [make(i) for i in range(layers)]
        g = torch.Generator(device="cuda").manual_seed(seed + layers)
        self.emb = torch.randn(vocab, hidden, device="cuda", generator=g).to(torch.bfloat16)
        self.head = W12Weight.from_device((torch.randn(vocab, hidden, device="cuda", generator=g) *
                                           hidden ** -0.5).to(torch.bfloat16))
        self.rope = rope_table(max_len, head_dim)
        self.selection = Beams(requests, beams, eos=eos)
        self.prefix = KVPrefix.create(requests, beams)
        self.copies = KVCopies.empty(self.rows)
        self.lens = torch.zeros(self.rows, dtype=torch.int32, device="cuda")
        self.new = torch.ones_like(self.lens)
        self.step = self.pages.step(self.rows)
        self.step.prefix = self.prefix
        self.stream = torch.cuda.Stream()
        self.logits = torch.zeros(self.rows, vocab, dtype=torch.bfloat16, device="cuda")

    def forward(self, tokens, step):
        x = self.emb[tokens]
        for block in self.blocks:
            x = block(x, step, self.rope)
        return x

    def vocabulary(self, x):
        return torch.cat([self.head.gemm(part) for part in x.split(MAX_TOKENS)])

    def begin(self, prompts):
        """The prompts' keys and values, and every beam's logits behind them."""
        new = torch.zeros_like(self.lens)
        new[::self.beams] = torch.tensor([len(p) for p in prompts], dtype=torch.int32)
        self.lens.zero_()
        step = self.pages.step(int(sum(map(len, prompts))), max_new=max(map(len, prompts)))
        self.pages.plan(self.lens, new, step)
        x = self.forward(torch.tensor([t for p in prompts for t in p], device="cuda"), step)
        first = self.vocabulary(x[step.cu_new[1:][::self.beams].long() - 1])
        self.logits.copy_(first.repeat_interleave(self.beams, 0))
        self.lens.copy_(new.view(-1, self.beams)[:, :1].expand(-1, self.beams).reshape(-1))
        self.selection.reset()

    def choose(self):
        """The beams that go on, in pages that they share."""
        self.selection.select(self.logits)
        self.pages.fork(self.selection.parents, self.lens, self.copies, prefix=self.prefix, lens_out=self.lens)
        self.blocks[0].cache.copy(self.copies, others=[b.cache for b in self.blocks[1:]])

    def decode(self):
        """The logits behind the chosen tokens.  (A beam that nothing goes on from has token -1
        and score -infinity; it goes along with any token.)"""
        self.pages.plan(self.lens, self.new, self.step)
        x = self.forward(self.selection.tokens.clamp(min=0).long(), self.step)
        self.logits.copy_(self.vocabulary(x))
        self.lens += 1

    def run(self, prompts, steps):
        """For each prompt its best hypotheses, (score, tokens, finished), best first: those that
        ended and the beams that are left after ``steps`` tokens."""
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):  # workspaces are a stream's: the graph's too
            history = self.search(prompts, steps)
        torch.cuda.current_stream().wait_stream(self.stream)
        w12.w12_check_status()
        history = [[t.tolist() for t in h] for h in history]

        def tokens_of(i, row):  # that the beam in `row` had after step i
            out = []
            for tokens, parents, *_ in history[i::-1] if i >= 0 else []:
                out.append(tokens[row])
                row = parents[row]
            return out[::-1]

        best = [[] for _ in prompts]
        for r, hyps in enumerate(best):
            for i, (tokens, parents, c_tokens, c_parents, c_scores, scores) in enumerate(history):
                for t, parent, score in zip(c_tokens[r], c_parents[r], c_scores[r]):
                    if t == self.selection.eos:
                        hyps.append((score, tokens_of(i - 1, parent) + [t], True))
            for k, score in enumerate(history[-1][-1][r]):
                if history[-1][0][r * self.beams + k] >= 0:
                    hyps.append((score, tokens_of(steps - 1, r * self.beams + k), False))
            hyps.sort(key=lambda h: -h[0])
            del hyps[self.beams:]
        return best

    def search(self, prompts, steps):
        """What every step's selection gave."""
        self.begin(prompts)
        history, graph = [], None
        for i in range(steps):
            if graph is None:
                if i > 0:
                    self.decode()
                self.choose()
                if i == 1:  # everything has had an ordinary call
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=self.stream):
                        self.decode()
                        self.choose()
            else:
                graph.replay()
            s = self.selection
            history.append([t.clone() for t in (s.tokens, s.parents, s.cand_tokens, s.cand_parents, s.cand_scores,
                                                s.scores)])
        return history

    def finish(self):
        """All pages go back."""
        self.pages.fork(torch.full_like(self.lens, -1), self.lens, self.copies, prefix=self.prefix, lens_out=self.lens)
        w12.w12_check_status()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=("bf16", "q8"), default="bf16")
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args()
    search = BeamSearch(a.requests, a.beams, cache=a.cache)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(1, 4001, (40 + 37 * r,), generator=g).tolist() for r in range(a.requests)]
    best = search.run(prompts, a.steps)
    shared = search.prefix.lens.view(a.requests, -1)[:, 0].tolist()
    held = int(search.pages.owned.sum())
    head, tail = search.pages.ring_state.tolist()
    used = search.pages.ring.numel() - (tail - head)
    search.finish()
    for r, hyps in enumerate(best):
        score, tokens, done = hyps[0]
        print(f"request {r}: {len(prompts[r])} tokens, {shared[r]} of them and of the answers shared; best score "
              f"{score:.2f}, {len(tokens)} tokens{' and ended' if done else ''}")
    print(f"{held} table entries in {used} pages, {a.cache} cache")


if __name__ == "__main__":
    main()
