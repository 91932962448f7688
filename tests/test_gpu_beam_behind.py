"""The beams that go on where they are not among the candidates asked for: selection keeps
enough of both, whichever tokens end."""
import math

import pytest
import torch
from test_gpu_beam import DTYPES, draw, pack, scores_ref

from lossless_bit_weight_encode_gb300 import Beams, w12

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def check_going_on(beams, ref, vocab):
    """tokens, parents and scores against the best of `ref` that do not end."""
    n, b = beams.requests, beams.beams
    tokens, parents, scores = (t.cpu().view(n, b) for t in (beams.tokens, beams.parents, beams.scores))
    for r in range(n):
        line = ref[r].clone()
        if beams.eos is not None and beams.eos < vocab:
            line.view(b, vocab)[:, beams.eos] = -INF
        order = line.sort(descending=True, stable=True)
        best, at = order.values[:b + 1].tolist(), order.indices[:b + 1].tolist()
        best += [-INF] * (b + 2 - len(best))
        seen = set()
        for i in range(b):
            if best[i] == -INF:
                assert (tokens[r, i], parents[r, i], scores[r, i]) == (-1, -1, -INF), (r, i)
                continue
            t, p = int(tokens[r, i]), int(parents[r, i]) - r * b
            assert 0 <= t < vocab and 0 <= p < b and t != beams.eos and (p, t) not in seen, (r, i)
            seen.add((p, t))
            # 4e-6 is the selection's own bound; the score is rounded to 32 bits
            near = 4e-6 + 2.0 ** -23 * abs(best[i])
            assert abs(float(line[p * vocab + t]) - best[i]) <= near, (r, i)
            assert abs(float(scores[r, i]) - best[i]) <= near, (r, i)
            if (i == 0 or best[i - 1] - best[i] > 2 * near) and best[i] - best[i + 1] > 2 * near:
                assert p * vocab + t == at[i], (r, i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [40, 9000])
@pytest.mark.parametrize("take", [1, 2, 5, 8, 30])
@pytest.mark.parametrize("rank", [0, 1, -1, 0.5, 1.5, None])
def test_the_token_that_ends_at_any_rank(rank, take, vocab, dtype):
    """`rank` 0 or 1: eos is the best or second token of all; -1 the last one asked for, 0.5 and
    1.5 the first and the beams-th behind; None: rare."""
    n, b = 3, 4
    logits, scores, _ = draw(n, b, vocab, dtype, 17 * take + vocab)
    ref = scores_ref(logits, scores, None).cpu()
    order = ref.sort(dim=1, descending=True, stable=True).indices
    at = {0: 0, 1: 1, -1: take - 1, 0.5: take, 1.5: take + b - 1}.get(rank)
    eos = vocab + 5 if rank is None else int(order[0, at]) % vocab
    beams = Beams(n, b, take=take, eos=eos)
    beams.select(logits, scores=scores)
    w12.w12_check_status()
    check_going_on(beams, ref, vocab)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("take", [1, 3, 16])
def test_every_beam_may_end(take, dtype):
    """eos is the best token of every beam: as many candidates as beams end."""
    n, b, vocab = 4, 8, 3000
    logits, scores, _ = draw(n, b, vocab, dtype, take)
    logits[:, 77] = 25.0
    ref = scores_ref(logits, scores, None).cpu()
    beams = Beams(n, b, take=take, eos=77)
    beams.select(logits, scores=scores)
    w12.w12_check_status()
    check_going_on(beams, ref, vocab)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("left", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("take", [1, 2, 9])
def test_fewer_than_beams(take, left, dtype):
    """`left` tokens that may go on in all beams of a request together, and eos in each."""
    n, b, vocab = 3, 4, 5000
    logits, scores, g = draw(n, b, vocab, dtype, 100 * take + left)
    allowed = torch.zeros(n * b, vocab, dtype=torch.bool, device="cuda")
    allowed[:, 4321] = True
    for i in range(left):
        allowed[torch.arange(n, device="cuda") * b + i % b, torch.randint(4000, (n,), device="cuda", generator=g)] = True
    beams = Beams(n, b, take=take, eos=4321)
    beams.select(logits, allowed=pack(allowed), scores=scores)
    w12.w12_check_status()
    check_going_on(beams, scores_ref(logits, scores, allowed).cpu(), vocab)
