"""Prompts behind a shared prefix (hundreds of new tokens per request, some of them more than a
row block has room for), against plain attention in 64 bits, and that calls repeat themselves."""
import pytest
import torch
from test_gpu_shared import compare, run, shared_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 2), (128, 12, 2), (128, 3, 3), (256, 6, 1)])
@pytest.mark.parametrize("groups,page", [
    ([(20, [(0, 300), (0, 33), (0, 129)]), (0, [(0, 64)])], 16),         # the first turn behind a system prompt
    ([(3, [(70, 300), (0, 1), (200, 0), (5, 511)])], 64),                # later turns, one of them decoding
    ([(1, [(None, 200), (40, 200)]), (2, [(0, 65), (None, 1)])], 48)])   # some of a group without the prefix
def test_prompts(groups, page, dim, heads, kv_heads, q8):
    compare(shared_case(groups, heads, kv_heads, dim, page, q8, seed=dim + heads))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("groups,heads", [([(90, [(50, 1)] * 8)] * 4, 48), ([(30, [(20, 1)] * 64)], 48),
                                          ([(5, [(0, 300)] * 3)], 12), ([(40, [(30, 4)] * 9)], 24)])
def test_calls_repeat_themselves(groups, heads, q8):
    cache, _, _, _, q, step = shared_case(groups, heads, heads // 6, 128, 64, q8, 41)
    first = [t.clone() for t in run(cache, q, step)]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, run(cache, q, step)))
