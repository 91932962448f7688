"""A whole beam search (selection, shared pages, their copies, attention behind the shared
prefix, part of it as a CUDA graph) against the same model over a cache of its own for
every hypothesis."""
import importlib.util
import os

import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVCache, KVPages, w12

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from gpu_util import ensure_built
    ensure_built()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")
    spec = importlib.util.spec_from_file_location("beam_search", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def check_pages(pages):
    """Every page is free or has its holders."""
    head, tail = pages.ring_state.tolist()
    ring = pages.ring.tolist()
    free = [ring[i % len(ring)] for i in range(head, tail)]
    holders = [0] * len(ring)
    for row, n in zip(pages.tables.tolist(), pages.owned.tolist()):
        for page in row[:n]:
            holders[page] += 1
    assert sorted(free + [p for p, n in enumerate(holders) if n]) == list(range(len(ring)))
    assert [max(n - 1, 0) for n in holders] == pages.shares.tolist()


def alone(search, prompt, tokens, cache):
    """The hypothesis's score with a cache and pages of its own, every token in a step of its
    own behind the prompt."""
    pages = KVPages.create(32, 16, 1, 32)
    caches = [b.cache for b in search.blocks]
    try:
        for b in search.blocks:
            c = b.cache
            b.cache = KVCache.empty(32, 16, c.kv_heads, c.head_dim, cache)
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        score, part = 0.0, prompt
        for t in tokens:
            step = pages.step(len(part), max_new=len(part))
            pages.plan(lens, torch.full_like(lens, len(part)), step)
            x = search.forward(torch.tensor(part, device="cuda"), step)
            score += float(search.vocabulary(x[-1:]).double().log_softmax(-1)[0, t])
            lens = lens + len(part)
            part = [t]
        w12.w12_check_status()
        return score
    finally:
        for b, c in zip(search.blocks, caches):
            b.cache = c


@pytest.mark.parametrize("requests,beams,cache,lengths,shape", [
    (1, 4, "bf16", [33], {}),
    (3, 5, "bf16", [1, 48, 77], dict(heads=8, kv_heads=4, head_dim=128)),
    (2, 8, "q8", [64, 19], {}),
    (2, 1, "bf16", [20, 5], {}),
])
def test_search_against_hypotheses_alone(example, requests, beams, cache, lengths, shape):
    steps = 11
    search = example.BeamSearch(requests, beams, vocab=601, max_len=128, cache=cache, seed=5, **shape)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(1, 601, (n,), generator=g).tolist() for n in lengths]
    best = search.run(prompts, steps)
    check_pages(search.pages)
    if beams > 1:  # full pages of the prompts are the beams' common prefix
        got = search.prefix.lens.view(requests, beams)
        for r, n in enumerate(lengths):
            if bool((search.selection.scores[r] > -1e30).all()):
                assert int(got[r].min()) >= n // 16 * 16
    for prompt, hyps in zip(prompts, best):
        assert len(hyps) == beams and all(a[0] >= b[0] for a, b in zip(hyps, hyps[1:]))
        assert len({tuple(t) for _, t, _ in hyps}) == beams
        for score, tokens, done in hyps:
            assert (tokens[-1] == 0) == done and 0 not in tokens[:-1]
            # Logits are up to about 4 and rounded to BF16 on both sides (2^-8 of them: 0.016
            # each, for the token and, less, for the sum over all); the roundings of two layers'
            # attention and sums (2^-8 of numbers about 1, for 512 columns with weights of
            # 512^-0.5 as many times the typical error) add as much again.
            assert abs(score - alone(search, prompt, tokens, cache)) <= 0.06 * len(tokens)
    search.finish()
    head, tail = search.pages.ring_state.tolist()
    assert tail - head == search.pages.ring.numel() and not int(search.pages.shares.abs().sum())


def test_a_second_search_over_the_same_pages(example):
    """The graph of one search, freed pages and old contents do not reach the next."""
    search = example.BeamSearch(2, 4, vocab=601, max_len=128, seed=7)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(1, 601, (n,), generator=g).tolist() for n in (30, 50)]
    first = search.run(prompts, 6)
    search.finish()
    search.run([p[::-1] for p in prompts], 5)
    check_pages(search.pages)
    search.finish()
    assert search.run(prompts, 6) == first
    check_pages(search.pages)
