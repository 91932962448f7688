"""Beam search's selection on the GPU, against the definition in 64 bits."""
import math

import pytest
import torch

from lossless_bit_weight_encode_gb300 import Beams, w12

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def pack(allowed):
    """[rows, vocab] of truth values as int32 words."""
    rows, vocab = allowed.shape
    words = -(-vocab // 32)
    bits = torch.zeros(rows, words * 32, dtype=torch.int64, device=allowed.device)
    bits[:, :vocab] = allowed
    v = (bits.view(rows, words, 32) << torch.arange(32, device=allowed.device)).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).to(torch.int32)


def scores_ref(logits, scores, allowed):
    """[requests, beams * vocab] scores in 64 bits; -infinity for what does not count."""
    n, b = scores.shape
    x = logits.double().view(n * b, -1)
    x = torch.where(torch.isnan(x), -INF, x)
    if allowed is not None:
        x = torch.where(allowed, x, -INF)
    m = x.amax(1, keepdim=True)
    d = torch.where(x == m, 0.0, x - m)
    d = torch.where((x == -INF) | torch.isnan(d), -INF, d)
    s = scores.double().reshape(n * b, 1) + (d - torch.log(torch.exp(d).sum(1, keepdim=True)))
    s = torch.where(torch.isfinite(scores).reshape(n * b, 1), s, -INF)
    return torch.where(torch.isnan(s), -INF, s).view(n, -1)


def check(beams, logits, scores, allowed=None, exact=False):
    """`exact`: the best ones are far apart, or equal in the same row."""
    n, b, take = beams.requests, beams.beams, beams.take
    vocab = logits.shape[-1]
    ref = scores_ref(logits, scores, allowed).cpu()
    order = torch.sort(ref, dim=1, descending=True, stable=True)
    deep = min(ref.shape[1], take + 2 * b + 4)
    best, at = order.values[:, :deep], order.indices[:, :deep]
    # each of a row's exponentials is off by 2^-22 and the argument's 2^-24 of at most 32:
    # 3e-6 of a sum, if all went the same way; the score itself is rounded to 32 bits
    tol = 4e-6
    ct, cp, cs = beams.cand_tokens.cpu().long(), beams.cand_parents.cpu().long(), beams.cand_scores.cpu().double()
    nt, np_, ns = (t.cpu().view(n, b) for t in (beams.tokens, beams.parents, beams.scores))
    nt, np_, ns = nt.long(), np_.long(), ns.double()
    for r in range(n):
        real = int((ref[r] > -INF).sum())
        for i in range(take):
            if i >= real:
                assert ct[r, i] == -1 and cp[r, i] == -1 and cs[r, i] == -INF
                continue
            place = (cp[r, i] - r * b) * vocab + ct[r, i]
            assert 0 <= ct[r, i] < vocab and r * b <= cp[r, i] < (r + 1) * b
            near = tol + 2.0 ** -23 * abs(float(best[r, i]))
            assert abs(float(ref[r, place] - best[r, i])) <= near or ref[r, place] == best[r, i]
            assert abs(float(cs[r, i] - ref[r, place])) <= near or cs[r, i] == ref[r, place].float()
            alone = all(j < 0 or j >= deep or j == i or abs(float(best[r, j] - best[r, i])) > 2 * near or
                        (best[r, j] == best[r, i] and at[r, j] // vocab == at[r, i] // vocab) for j in (i - 1, i + 1))
            if exact or alone:
                assert place == at[r, i], (r, i)
            if i and cp[r, i - 1] == cp[r, i]:  # in a row: by the logits, then by the token
                x, y = ref[r, (cp[r, i] - r * b) * vocab + ct[r, i - 1]], ref[r, place]
                assert x > y or (x == y and ct[r, i - 1] < ct[r, i])
        assert len({(int(p), int(t)) for p, t in zip(cp[r], ct[r]) if t >= 0}) == min(real, take)
        # the beams that go on: the candidates in order, without those that end
        kept = [(int(t), int(p), float(s)) for t, p, s in zip(ct[r], cp[r], cs[r]) if t >= 0 and t != beams.eos]
        got = [(int(t), int(p), float(s)) for t, p, s in zip(nt[r], np_[r], ns[r])]
        upto = min(len(kept), b)
        assert got[:upto] == kept[:upto]
        if take >= real or len(kept) >= b:
            assert got[upto:] == [(-1, -1, -INF)] * (b - upto)
        assert all(t != beams.eos for t, _, _ in got if beams.eos is not None)


def run(logits, scores, allowed=None, take=None, eos=None, exact=False, line=False):
    n, b = scores.shape
    beams = Beams(n, b, take=take, eos=eos)
    words = None if allowed is None else pack(allowed[:1])[0].contiguous() if line else pack(allowed)
    beams.select(logits, allowed=words, scores=scores)
    torch.cuda.synchronize()
    w12.w12_check_status()
    check(beams, logits, scores, allowed, exact)
    return beams


def draw(n, b, vocab, dtype, seed, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(n * b, vocab, device="cuda", generator=g) * spread).to(dtype)
    scores = -torch.rand(n, b, device="cuda", generator=g) * 4
    return logits, scores, g


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,b,vocab", [(1, 1, 1), (1, 4, 3), (2, 3, 31), (3, 2, 1000), (2, 5, 4097), (1, 32, 8191),
                                       (5, 8, 33001), (1, 4, 151936), (40, 1, 2049), (3, 16, 50257)])
@pytest.mark.parametrize("eos", [False, True])
def test_select(n, b, vocab, dtype, eos):
    logits, scores, _ = draw(n, b, vocab, dtype, vocab + b)
    end = vocab // 2 if eos else None
    if eos:
        logits[::2, end] = 20.0
    run(logits, scores, eos=end)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("take", [1, 7, 9, 17, 33, 64])
def test_take(take, dtype):
    logits, scores, _ = draw(3, 4, 9000, dtype, take)
    run(logits, scores, take=take, eos=5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("density", [0.0, 0.0005, 0.1, 0.9])
def test_allowed(density, dtype):
    logits, scores, g = draw(4, 3, 20011, dtype, 5)
    allowed = torch.rand(logits.shape, device="cuda", generator=g) < density
    allowed[1] = False                     # a row that nothing is left of
    allowed[2] = False
    allowed[2, 20010] = True               # the last token alone
    allowed[3] = False
    allowed[3, 7000:8100] = True           # a run of tokens
    logits[~allowed] = float("nan")        # what does not count has no effect
    run(logits, scores, allowed)
    run(logits[:, 1:], scores, allowed[:, 1:])  # rows that begin anywhere
    run(logits, scores, allowed[:1].expand_as(allowed), line=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [700, 8000, 40000])
@pytest.mark.parametrize("kind", ["equal", "steps", "rising", "falling", "lumps", "zeros"])
def test_orders_that_are_not_random(kind, vocab, dtype):
    b = 3
    at = torch.arange(vocab, device="cuda", dtype=torch.float64)
    x = {"equal": torch.zeros_like(at), "steps": (at % 7).floor(), "rising": at / vocab * 40, "falling": -at / vocab * 40,
         "lumps": torch.where((at // 8) % 256 == 3, 5.0, 0.0) + (at % 8) / 16,  # all of a thread's elements, and few threads
         "zeros": torch.where(at % 2 == 0, -0.0, 0.0)}[kind]
    logits = x.to(dtype).expand(2 * b, -1).contiguous()
    scores = torch.tensor([[0.0, -9.5, -3.25], [-1.0, -1.0, -1.0]], device="cuda")
    run(logits, scores, exact=True)
    run(logits, scores, take=64, exact=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [9000, 20011, 70003])
@pytest.mark.parametrize("kind", ["random", "equal", "rising", "one tile", "mask"])
def test_many_rows_of_several_tiles(kind, vocab, dtype):
    """More rows than the device has places for, so that a block takes several tiles."""
    n, b = 80, 8
    at = torch.arange(vocab, device="cuda", dtype=torch.float64)
    logits, scores, g = draw(n, b, vocab, dtype, vocab)
    allowed = None
    if kind == "equal":
        logits.zero_()
    elif kind == "rising":
        logits.copy_((at / vocab * 40).expand_as(logits))
    elif kind == "one tile":
        logits[:, vocab - 700:] += 30  # all that counts in the last one
    elif kind == "mask":
        allowed = torch.rand(logits.shape, device="cuda", generator=g) < 0.01
        allowed[:, :8200] = False  # a first tile without tokens
        logits[~allowed] = float("inf")
    run(logits, scores, allowed, eos=vocab - 1, exact=kind in ("equal", "rising"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_that_are_not_finite(dtype):
    logits, scores, _ = draw(5, 2, 5000, dtype, 8)
    low = torch.finfo(dtype).min
    logits[0, 100:110] = INF          # share the weight
    logits[1] = float("nan")          # nothing left
    logits[2, 50:] = -INF             # fifty left
    logits[3] = float("nan")
    logits[3, 4999] = -7.0            # one left
    logits[4] = low                   # masked by the type's lowest value, all of it
    logits[5, 4:] = low               # but for four
    logits[6] = torch.finfo(dtype).max
    logits[7, ::3] = -INF
    run(logits, scores)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_logits(dtype):
    logits, scores, _ = draw(2, 2, 30000, dtype, 8, spread=1.0)
    logits[0] *= 1e5
    logits[1] *= 1e8       # beyond what whole powers of two are exact for
    logits[2] -= 3e7
    logits[3] *= 1e30
    run(logits, scores)


def test_beams_that_do_not_go_on():
    logits, scores, _ = draw(4, 4, 6000, torch.bfloat16, 1)
    scores[0, 1:] = -INF
    scores[1] = -INF
    scores[2, 0], scores[2, 3] = float("nan"), INF
    logits[2] = float("nan")
    run(logits, scores, eos=3)


def test_search_in_place_over_steps():
    n, b, vocab = 3, 4, 3001
    beams = Beams(n, b, eos=17)
    scores = torch.full((n, b), -INF, device="cuda")
    scores[:, 0] = 0
    for i in range(5):
        logits, _, _ = draw(n, b, vocab, torch.bfloat16, 50 + i)
        beams.select(logits)
        torch.cuda.synchronize()
        check(beams, logits, scores)
        scores = beams.scores.clone()
    beams.reset()
    assert beams.scores[:, 0].tolist() == [0.0] * n and torch.isinf(beams.scores[:, 1:]).all()


def test_layouts():
    logits, scores, _ = draw(2, 3, 5003, torch.bfloat16, 3)
    wide = torch.zeros(6, 6000, device="cuda", dtype=torch.bfloat16)
    for off in (0, 1, 5, 8):
        view = wide[:, off:off + 5003]
        view.copy_(logits)
        run(view, scores)
    wide = torch.zeros(6, 6000, device="cuda")
    for off in (0, 1, 2, 3):
        view = wide[:, off:off + 5003]
        view.copy_(logits)
        run(view, scores)
    beams = Beams(2, 3)
    beams.select(logits.view(2, 3, 5003), scores=scores)
    torch.cuda.synchronize()
    check(beams, logits, scores)


def test_same_results_every_time_and_other_vocabularies():
    logits, scores, _ = draw(8, 4, 70000, torch.float32, 2)
    small, _, _ = draw(8, 4, 900, torch.bfloat16, 2)
    beams = Beams(8, 4)
    first = None
    for _ in range(20):
        beams.select(small, scores=scores)
        check(beams, small, scores)
        beams.select(logits, scores=scores)
        got = (beams.cand_tokens.clone(), beams.cand_parents.clone(), beams.cand_scores.clone())
        first = first or got
        assert all(torch.equal(a, c) for a, c in zip(first, got))
    check(beams, logits, scores)


def test_stream_and_graph():
    logits, scores, _ = draw(2, 4, 20000, torch.bfloat16, 4)
    beams = Beams(2, 4)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    beams.select(logits, scores=scores, stream=stream)
    stream.synchronize()
    check(beams, logits, scores)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beams.select(logits, scores=scores)
    for seed in (6, 7):
        logits.copy_(draw(2, 4, 20000, torch.bfloat16, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        check(beams, logits, scores)
    fresh = Beams(2, 4)
    with pytest.raises(RuntimeError, match="ordinary call"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            fresh.select(logits, scores=scores)


def test_refusals():
    for bad in (dict(requests=0, beams=1), dict(requests=1, beams=33), dict(requests=1, beams=2, take=65),
                dict(requests=1, beams=2, take=0), dict(requests=1, beams=2, eos=-1)):
        with pytest.raises(ValueError):
            Beams(**bad)
    beams = Beams(2, 2)
    x, _, _ = draw(2, 2, 100, torch.bfloat16, 0)
    words = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=x[:3]), dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x.t()),
                dict(logits=x.view(2, 2, 100).transpose(0, 1)), dict(logits=x[0]),
                dict(allowed=words[:, :3]), dict(allowed=words[:2]), dict(allowed=words.long()),
                dict(allowed=words.t()), dict(allowed=words[0, :3]), dict(scores=torch.zeros(3, device="cuda")),
                dict(scores=torch.zeros(2, 2, device="cuda").double()), dict(scores=torch.zeros(2, 2))):
        with pytest.raises(ValueError):
            beams.select(**{**dict(logits=x), **bad})
    with pytest.raises(TypeError):
        beams.select([1.0])
    with pytest.raises(AttributeError):
        beams.tokens = words
