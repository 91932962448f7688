"""Paged-cache calls at the ends of their ranges: calls that run longer than the limit of
their waits, and tables of close to 2^31 entries."""
import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVCache, KVPages, KVStep, w12
from test_gpu_kv import check_attend, dev, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def some_rows(q, cache, count, rows, group):
    """attend_ref for chosen tokens of one request without a past, pages in order."""
    dim, hk = q.shape[2], cache.kv_heads
    k, v = (t.transpose(1, 2).reshape(-1, hk, dim)[:count].double() for t in (cache.k, cache.v))
    got = [[], [], [], []]
    for i in rows:
        row = q[i].double().view(hk, group, dim)
        s = torch.einsum("hgd,khd->hgk", row, k[:i + 1]) * dim ** -0.5
        p = torch.softmax(s, -1)
        big = (torch.einsum("hgd,khd->hgk", row.abs(), k[:i + 1].abs()) * dim ** -0.5).amax(-1)
        for a, x in zip(got, (torch.einsum("hgk,khd->hgd", p, v[:i + 1]), torch.logsumexp(s, -1),
                              torch.einsum("hgk,khd->hgd", p, v[:i + 1].abs()), big)):
            a.append(x.reshape(-1, *x.shape[2:]).cpu())
    return tuple(torch.stack(x) for x in got)


# rows that take the tcgen05 kernel, and (by the count that the caller gives) the warp-level one
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,max_new", [(40000, 48, 8, 128, 40000), (60000, 8, 4, 64, 1)])
def test_call_longer_than_the_limit(w12_opts, tokens, heads, kv_heads, dim, max_new):
    """The limit grows with a call's work: a long prompt's may take many times timeout_ms."""
    limit_ms = 10
    page, pages = 64, -(-tokens // 64)
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    cache = KVCache(rnd(pages, kv_heads, page, dim), rnd(pages, kv_heads, page, dim))
    step = KVStep(torch.arange(pages, dtype=torch.int32, device="cuda")[None], dev([0], torch.int32),
                  dev([0, tokens], torch.int32), max_new=max_new)
    q, lse = rnd(tokens, heads, dim), torch.empty(tokens, heads, device="cuda")
    out = torch.empty(tokens, heads * dim, device="cuda", dtype=torch.bfloat16)
    cache.attend(q[:1].view(1, -1), KVStep(step.tables, step.lens, dev([0, 1], torch.int32)))  # set-up
    status()
    w12_opts(timeout_ms=limit_ms)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    cache.attend(q.view(tokens, -1), step, out=out, lse=lse)
    end.record()
    status()
    assert start.elapsed_time(end) > 3 * limit_ms, "the case is too short for what it tests"
    rows = [0, 1, 127, 5000, tokens // 2, tokens - 1]
    check_attend(out[rows].view(len(rows), heads, dim), lse[rows], some_rows(q, cache, tokens, rows, heads // kv_heads))


def test_plan_of_nearly_two_to_the_31_table_entries():
    """More than 2^31 - 1024 pages are taken in one call; all but five are missing."""
    requests, blocks, page = 16, (1 << 27) - 1, 16
    tables = torch.full((requests, blocks), 7, dtype=torch.int32, device="cuda")
    pages = KVPages(tables, torch.zeros(requests, dtype=torch.int32, device="cuda"), dev([30, 31, 32, 33, 34], torch.int32),
                    dev([1, 6], torch.int64), page)
    lens = torch.full((requests,), blocks * page, dtype=torch.int32, device="cuda")
    step = pages.step(4096)
    pages.plan(lens, torch.zeros_like(lens), step)
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 3
    assert tables[0, :6].tolist() == [31, 32, 33, 34, 30, -1]
    assert pages.owned.tolist() == [5] + [0] * 15 and pages.ring_state.tolist() == [6, 6]
    tables[0, :5] = -1
    assert all(bool((row == -1).all()) for row in tables)
