"""What beam search's selection gives exactly: the score of a token that alone counts, and equal
scores for rows whose logits differ by a constant."""
import math

import pytest
import torch
from test_gpu_beam import DTYPES, draw, pack

from lossless_bit_weight_encode_gb300 import Beams, w12

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def select(logits, scores, allowed=None, **kw):
    beams = Beams(*scores.shape, **kw)
    beams.select(logits, allowed=allowed, scores=scores)
    w12.w12_check_status()
    return beams


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 40, 5000, 151936])
def test_a_token_that_alone_counts_keeps_the_score(vocab, dtype):
    """ln 1 is 0: the score is the beam's own, and equal ones go to the lower beam."""
    n, b = 24, 7
    logits, _, g = draw(n, b, vocab, dtype, vocab, spread=9.0)
    token = torch.randint(vocab, (n * b,), device="cuda", generator=g)
    allowed = torch.zeros(n * b, vocab, dtype=torch.bool, device="cuda")
    allowed[torch.arange(n * b, device="cuda"), token] = True
    scores = (-5 * torch.rand(n, 1, device="cuda", generator=g)).expand(n, b).contiguous()
    scores[::2] = 0.0
    beams = select(logits, scores, pack(allowed))
    rows = torch.arange(n * b, dtype=torch.int32, device="cuda")
    assert torch.equal(beams.scores, scores)
    assert torch.equal(beams.parents, rows) and torch.equal(beams.tokens, token.int())
    assert torch.equal(beams.cand_scores[:, :b], scores)
    scores = -5 * torch.rand(n, b, device="cuda", generator=g)
    beams = select(logits, scores, pack(allowed))
    assert torch.equal(beams.scores, scores.sort(dim=1, descending=True).values)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("vocab", [9, 3000, 151936])
@pytest.mark.parametrize("kind", ["equal", "two", "few", "many", "rising"])
def test_rows_that_differ_by_a_constant_have_equal_scores(kind, vocab, n, dtype):
    """Their softmax is the same: what both give goes to the lower beam.  All logits are
    multiples of 1/8 below 16 (7 bits), so that the constants can be added without rounding."""
    b, take = 4, 13
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randint(-40, 41, (n, 1, vocab), device="cuda", generator=g) / 8.0
    if kind == "equal":
        x.zero_()
    elif kind == "two":  # two tokens have nearly all of the weight
        x -= 6
        x[..., 0], x[..., vocab - 1] = 7.0, 6.625
    elif kind == "few":
        x = torch.where(x >= 4.875, x + 2, x - 5)
    elif kind == "rising":  # the maximum changes from tile to tile
        x = (torch.arange(vocab, device="cuda", dtype=torch.float64) / vocab * 80).floor().float().view(1, 1, -1) / 8 - 5
        x = x.expand(n, 1, vocab)
    shift = torch.tensor([0.0, 3.0, -4.0, 1.125], device="cuda").view(1, b, 1)
    logits = (x + shift).to(dtype)
    assert torch.equal(logits.float() - shift, x.expand(n, b, vocab))
    scores = torch.full((n, b), -1.75, device="cuda")
    beams = select(logits.view(n * b, vocab), scores, take=take)
    order = x[:, 0].sort(dim=1, descending=True, stable=True).indices
    token = torch.full((n, take), -1, dtype=torch.int64, device="cuda")
    parent = token.clone()
    for r in range(n):  # by value, then beam, then token
        value = x[r, 0][order[r]]
        line = []
        for v in value.unique(sorted=True).flip(0).tolist():
            same = order[r][value == v][:take].tolist()
            line += [(r * b + beam, t) for beam in range(b) for t in same]
            if len(line) >= take:
                break
        for i, (p, t) in enumerate(line[:take]):
            parent[r, i], token[r, i] = p, t
    assert torch.equal(beams.cand_parents.long(), parent) and torch.equal(beams.cand_tokens.long(), token)
    for r in range(n):  # bit by bit the same for equal logits
        v = torch.where(token[r] >= 0, x[r, 0][token[r].clamp(min=0)], -INF)
        for i in range(1, min(take, int((token[r] >= 0).sum()))):
            assert (beams.cand_scores[r, i] == beams.cand_scores[r, i - 1]) == (v[i] == v[i - 1])
