"""The C ABI's calls for shared pages, shared prefixes and beam search refuse bad arguments
before they touch a device (no GPU needed)."""
import ctypes

import pytest
from test_kv_host import BAD_CACHES, attend, cache

from lossless_bit_weight_encode_gb300 import build as libbuild
from lossless_bit_weight_encode_gb300 import w12

INVALID, SHAPE, ALIGN = 1, 2, 4
A = 1 << 20  # an aligned address that no call here gets to use


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def fork(**kw):
    f = {n: A for n in ("parents", "lens", "lens_out", "owned", "tables", "ring", "ring_state", "shares", "src", "dst",
                        "rows", "prefix_cu", "prefix_lens")}
    f.update(table_stride=8, num_pages=9, requests=2, max_blocks=8, page_size=16, ring_size=10, groups=1)
    f.update(kw)
    return w12.w12_kv_fork_args(**f)


def beam(**kw):
    f = dict(logits=A, logits_stride=100, allowed=None, allowed_stride=0, scores_in=A, scores=A, tokens=A, parents=A,
             cand_tokens=A, cand_parents=A, cand_scores=A, requests=2, beams=3, vocab=100, take=6, eos=-1,
             dtype=w12.BEAM_BF16)
    f.update(kw)
    return w12.w12_beam_args(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(requests=0), INVALID), (dict(max_blocks=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(prefix_cu=None), INVALID), (dict(prefix_lens=None), INVALID), (dict(groups=0), INVALID),
    (dict(groups=3), SHAPE), (dict(requests=4097), SHAPE), (dict(ring_size=8), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=24), SHAPE), (dict(table_stride=7), SHAPE),
    (dict(max_blocks=1 << 27, table_stride=1 << 27), SHAPE), (dict(lens=A + 2), ALIGN), (dict(shares=A + 1), ALIGN),
    (dict(ring_state=A + 4), ALIGN), (dict(prefix_lens=A + 2), ALIGN)] +
    [({n: None}, INVALID) for n in ("parents", "lens", "owned", "tables", "ring", "ring_state", "shares", "src", "dst",
                                    "rows")])
def test_fork_refused(kw, status):
    assert w12.lib().w12_kv_fork(fork(**kw), A, 1 << 30, None) == status
    assert w12.w12_last_error() != ""


def test_fork_null():
    L, size = w12.lib(), ctypes.c_size_t()
    assert L.w12_kv_fork(None, A, 1 << 30, None) == INVALID
    assert L.w12_kv_fork(fork(), None, 1 << 30, None) == INVALID
    assert L.w12_kv_fork(fork(), A + 64, 1 << 30, None) == ALIGN
    assert L.w12_kv_fork_workspace_size(fork(), None) == INVALID
    assert L.w12_kv_fork_workspace_size(None, ctypes.byref(size)) == INVALID
    assert L.w12_kv_fork_workspace_size(fork(requests=4097), ctypes.byref(size)) == SHAPE


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_caches_refused(kw, status):
    L, c, size = w12.lib(), cache(**kw), ctypes.c_size_t()
    prefix = w12.w12_kv_prefix(A, A, 1, 2)
    assert L.w12_kv_copy(c, 1, A, A, None, 1, None) == status
    assert L.w12_kv_attend_shared(c, attend(), prefix, A, 1 << 30, None) == status
    assert L.w12_kv_attend_shared_workspace_size(c, attend(), prefix, ctypes.byref(size)) == status


def test_copy_refused():
    L = w12.lib()
    two = (w12.w12_kv_cache * 2)(cache(), cache(num_pages=5))
    assert L.w12_kv_copy(two, 2, A, A, None, 1, None) == SHAPE
    two = (w12.w12_kv_cache * 2)(cache(), cache(dtype=w12.KV_Q8, scales_dev=A))
    assert L.w12_kv_copy(two, 2, A, A, None, 1, None) == SHAPE
    two = (w12.w12_kv_cache * 2)(cache(), cache(k_dev=None))
    assert L.w12_kv_copy(two, 2, A, A, None, 1, None) == INVALID
    assert L.w12_kv_copy(None, 1, A, A, None, 1, None) == INVALID
    assert L.w12_kv_copy(cache(), 0, A, A, None, 1, None) == INVALID
    assert L.w12_kv_copy(cache(), 1, None, A, None, 1, None) == INVALID
    assert L.w12_kv_copy(cache(), 1, A, None, None, 1, None) == INVALID
    assert L.w12_kv_copy(cache(), 1, A, A, None, -1, None) == INVALID
    assert L.w12_kv_copy(cache(), 1, A, A, A + 2, 1, None) == ALIGN
    assert L.w12_kv_copy(cache(), 1, A + 1, A, None, 1, None) == ALIGN


@pytest.mark.parametrize("kw,prefix,status", [
    (dict(window=4), (A, A, 1, 2), INVALID), ({}, (A, A, 0, 2), INVALID), ({}, (A, A, 1, -1), INVALID),
    ({}, (None, A, 1, 2), INVALID), ({}, (A, None, 1, 2), INVALID), ({}, (A, A, 3, 2), SHAPE),
    ({}, (A + 2, A, 1, 2), ALIGN), ({}, (A, A + 1, 1, 2), ALIGN), (dict(heads=3), (A, A, 1, 2), SHAPE),
    (dict(q=None), (A, A, 1, 2), INVALID), (dict(out=A + 2), (A, A, 1, 2), ALIGN),
    (dict(q_stride=248), (A, A, 1, 2), SHAPE)])
def test_attend_shared_refused(kw, prefix, status):
    L = w12.lib()
    assert L.w12_kv_attend_shared(cache(), attend(**kw), w12.w12_kv_prefix(*prefix), A, 1 << 30, None) == status


def test_attend_shared_null():
    L, p = w12.lib(), w12.w12_kv_prefix(A, A, 1, 2)
    assert L.w12_kv_attend_shared(cache(), attend(), None, A, 1 << 30, None) == INVALID
    assert L.w12_kv_attend_shared(cache(), None, p, A, 1 << 30, None) == INVALID
    assert L.w12_kv_attend_shared(cache(), attend(), p, None, 1 << 30, None) == INVALID
    assert L.w12_kv_attend_shared(cache(), attend(), p, A + 128, 1 << 30, None) == ALIGN
    assert L.w12_kv_attend_shared_workspace_size(cache(), attend(), p, None) == INVALID


BAD_BEAMS = [(dict(requests=0), INVALID), (dict(beams=0), INVALID), (dict(vocab=0), INVALID), (dict(take=0), INVALID),
             (dict(eos=-2), INVALID), (dict(dtype=2), INVALID), (dict(beams=33), SHAPE), (dict(take=65), SHAPE),
             (dict(vocab=(1 << 22) + 1), SHAPE), (dict(requests=1 << 28, beams=32), SHAPE)]


@pytest.mark.parametrize("kw,status", BAD_BEAMS + [
    (dict(logits_stride=99), SHAPE), (dict(allowed=A, allowed_stride=3), SHAPE), (dict(logits=A + 1), ALIGN),
    (dict(dtype=w12.BEAM_F32, logits=A + 2), ALIGN), (dict(allowed=A + 2), ALIGN), (dict(scores=A + 2), ALIGN),
    (dict(cand_parents=A + 1), ALIGN)] +
    [({n: None}, INVALID) for n in ("logits", "scores_in", "scores", "tokens", "parents", "cand_tokens",
                                    "cand_parents", "cand_scores")])
def test_beam_refused(kw, status):
    assert w12.lib().w12_beam_select(beam(**kw), A, 1 << 30, None) == status
    assert w12.w12_last_error() != ""


@pytest.mark.parametrize("kw,status", BAD_BEAMS)
def test_beam_workspace_refused(kw, status):
    size = ctypes.c_size_t()
    assert w12.lib().w12_beam_workspace_size(beam(**kw), ctypes.byref(size)) == status


def test_beam_null():
    L = w12.lib()
    assert L.w12_beam_select(None, A, 1 << 30, None) == INVALID
    assert L.w12_beam_select(beam(), None, 1 << 30, None) == INVALID
    assert L.w12_beam_select(beam(), A + 64, 1 << 30, None) == ALIGN
    assert L.w12_beam_workspace_size(beam(), None) == INVALID
