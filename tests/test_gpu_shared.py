"""Attention behind shared prefixes on the GPU, against plain attention in 64 bits over each
request's whole table."""
import random
import threading

import numpy as np
import pytest
import torch
from test_gpu_kv import attend_ref, check_attend, dev, make_cache, status

from lossless_bit_weight_encode_gb300 import KVPrefix, KVStep, w12

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def shared_case(groups, heads, kv_heads, dim, page, q8, seed, layout="hnd", stale=True, spare=3):
    """groups: a list of (prefix pages, [(own cached tokens, new tokens)]); a member with own
    None is empty: no prefix, nothing cached."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = 0
    for ahead, members in groups:
        need += ahead + sum(-(-((own or 0) + new) // page) for own, new in members)
    cache = make_cache(need + spare, kv_heads, page, dim, q8, layout)
    if q8:
        for t in (cache.k, cache.v):
            t.copy_(torch.randint(-127, 128, t.shape, device="cuda", generator=g, dtype=torch.int8))
        cache.scales.copy_(torch.rand(cache.scales.shape, device="cuda", generator=g) * 0.01 + 0.005)
    else:
        for t in (cache.k, cache.v):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
    ids = list(rng.permutation(need + spare))
    tables, lens, cu, pcu, plens, most = [], [], [0], [0], [], 1
    for ahead, members in groups:
        first = [ids.pop() for _ in range(ahead)]
        for own, new in members:
            alone = own is None
            mine = [ids.pop() for _ in range(-(-((own or 0) + new) // page))]
            tables.append(([] if alone else first) + mine)
            lens.append(0 if alone else ahead * page + own)
            plens.append(0 if alone else ahead * page)
            cu.append(cu[-1] + new)
            left = (own or 0) + new - (len(mine) - 1) * page
            if stale and mine and left < page:
                for t in (cache.scales,) if q8 else (cache.k, cache.v):
                    t[int(mine[-1]), :, left:] = float("nan")
        pcu.append(len(lens))
        most = max(most, len(members))
    width = max(len(t) for t in tables) + 1
    tables = np.array([t + [-1] * (width - len(t)) for t in tables], np.int64)
    q = torch.randn(max(cu[-1], 1), heads, dim, device="cuda", generator=g).to(torch.bfloat16)[:cu[-1]]
    prefix = KVPrefix(dev(pcu, torch.int32), dev(plens, torch.int32), max_requests=most)
    step = KVStep(dev(tables.tolist(), torch.int32), dev(lens, torch.int32), dev(cu, torch.int32),
                  max_new=max(n for _, m in groups for _, n in m), prefix=prefix)
    return cache, tables, lens, cu, q, step


def run(cache, q, step, **kw):
    t, h, d = q.shape
    lse = torch.full((t, h), 7.0, device="cuda")
    out = cache.attend(q.reshape(t, h * d), step, lse=lse, **kw)
    status()
    return out, lse


def compare(case, tree=None, scale=None):
    cache, tables, lens, cu, q, step = case
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse = run(cache, q, step, scale=scale)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, tree, 0, scale, q.shape[1] // cache.kv_heads))
    return out, lse


HEADS = [(64, 8, 8), (64, 8, 1), (128, 12, 2), (128, 5, 1), (256, 6, 1), (256, 4, 2), (128, 33, 1), (64, 20, 1)]
SHAPES = [
    ([(1, [(0, 1), (0, 1)])], 16),                                            # own tokens: the new one alone
    ([(7, [(3, 1), (40, 1), (17, 1), (0, 1)])], 16),                          # four beams
    ([(3, [(5, 1), (100, 2), (64, 1)]), (0, [(9, 1), (0, 3)]), (2, [(1, 1)])], 48),  # groups that share nothing, and one alone
    ([(2, [(3, 1)] * 30), (5, [(70, 1)] * 13)], 32),                          # more rows than a row block
    ([(4, [(6, 4), (None, 1), (11, 0), (0, 5)]), (1, [(None, 2), (200, 1)])], 64),  # empty members, some without new tokens
]


@pytest.mark.parametrize("dim,heads,kv_heads", HEADS)
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("groups,page", SHAPES)
def test_attend_shared(dim, heads, kv_heads, q8, groups, page):
    compare(shared_case(groups, heads, kv_heads, dim, page, q8, seed=dim + heads + page))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads,new", [(64, 4, 2, 1), (128, 12, 2, 1), (256, 2, 1, 1), (128, 12, 2, 3)])
def test_long_prefix_split_over_ctas(dim, heads, kv_heads, new, q8):
    compare(shared_case([(180, [(500, new), (31, new), (0, 1)]), (33, [(2000, 1), (7, new)])], heads, kv_heads, dim, 64,
                        q8, seed=dim))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 4), (128, 12, 2), (256, 6, 1)])
def test_trees(q8, dim, heads, kv_heads):
    groups = [(3, [(0, 6), (33, 16), (5, 32)]), (1, [(7, 1), (8, 4)])]
    case = shared_case(groups, heads, kv_heads, dim, 16, q8, seed=dim + heads)
    rng = random.Random(dim)
    masks = []
    for _, members in groups:
        for _, n in members:
            m = []
            for i in range(n):
                m.append((m[rng.randrange(i)] if i else 0) | 1 << i)
            masks += m
    masks[0] = 0           # sees the prefix alone
    masks[2] = 1 << 5      # a later token, and not itself
    masks[7] = 0xFFFFFFFF  # bits behind the request's last token
    tree = np.array(masks, np.uint32).view(np.int32)
    case[-1].tree = torch.from_numpy(tree).cuda()
    compare(case, tree=tree)


@pytest.mark.parametrize("layout", ["nhd", "gap"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layouts_and_strided_q(layout, q8, dim):
    cache, tables, lens, cu, q, step = shared_case([(3, [(20, 1), (0, 2)]), (1, [(5, 1)])], 6, 2, dim, 32, q8, 5, layout)
    t = q.shape[0]
    wide = torch.zeros(t, 8 * dim + 16, device="cuda", dtype=torch.bfloat16)
    rows = wide[:, 8:8 + 6 * dim]
    rows.copy_(q.view(t, -1))
    out = torch.full((t + 2, 6 * dim), 3.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.zeros(t, 6, device="cuda")
    assert cache.attend(rows, step, out=out[:t], lse=lse).data_ptr() == out.data_ptr()
    status()
    check_attend(out[:t], lse, attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, 3))
    assert (out[t:] == 3).all()


@pytest.mark.parametrize("members", [2, 11])
@pytest.mark.parametrize("q8", [False, True])
def test_absent_pages(members, q8):
    case = shared_case([(5, [(40, 1)] * members), (2, [(3, 1), (70, 2)])], 12, 2, 128, 16, q8, 4)
    cache, tables, _, _, _, step = case
    tables[:members, 2] = -1              # a hole in the prefix
    tables[0, 5] = cache.k.shape[0] + 7   # and in a request's own pages
    tables[members, :2] = -1              # a prefix that is not there at all
    tables[members + 1, :2] = -1
    step.tables = dev(tables.tolist(), torch.int32)
    compare(case)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("heads,members", [(2, 3), (12, 3), (12, 9)])
def test_values_that_are_not_finite(bad, heads, members):
    """One in the prefix reaches all of the group's requests, one of a request's own only it,
    and none another group."""
    groups = [(30, [(20, 1)] * members), (4, [(10, 1), (0, 1)])]
    case = shared_case(groups, heads, 1, 128, 16, False, 6)
    cache, tables, lens, cu, q, step = case
    clean, _ = run(cache, q, step)
    cache.v[int(tables[0, 11]), 0, 3, 5] = bad
    cache.v[int(tables[1, 30]), 0, 2, 9] = bad
    out, _ = run(cache, q, step)
    out, clean = (t.view(len(lens), heads, 128) for t in (out, clean))
    assert (~torch.isfinite(out[:members, :, 5])).all() and (~torch.isfinite(out[1, :, 9])).all()
    touched = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    touched[:members, :, 5] = True
    touched[1, :, 9] = True
    assert torch.equal(out[~touched], clean[~touched])
    cache.k[int(tables[0, 4]), 0, 1] = float("nan")  # a key: the group's rows
    out, lse = run(cache, q, step)
    out = out.view(len(lens), heads, 128)
    assert torch.isnan(out[:members]).all() and torch.isnan(lse[:members]).all()
    assert torch.equal(out[members:], clean[members:])


@pytest.mark.parametrize("scale", [5.0, -0.7, 0.0])
@pytest.mark.parametrize("heads", [4, 24])
def test_scales(scale, heads):
    compare(shared_case([(9, [(33, 1), (2, 1)])], heads, 2, 128, 32, False, 7), scale=scale)


def test_rows_of_no_request_are_left():
    cache, tables, lens, cu, q, step = shared_case([(2, [(5, 1), (9, 1)])], 4, 2, 64, 16, False, 8)
    more = torch.cat([q, q, q])
    out = torch.full((6, 256), 5.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((6, 4), 6.0, device="cuda")
    cache.attend(more.view(6, 256), step, out=out, lse=lse)
    status()
    check_attend(out[:2], lse[:2], attend_ref(q, cache, tables, lens, cu, None, 0, 0.125, 2))
    assert (out[2:] == 5).all() and (lse[2:] == 6).all()


def test_more_requests_than_max_says():
    case = shared_case([(3, [(5, 1)] * 9)], 6, 1, 128, 16, False, 9)
    case[-1].prefix.max_requests = 1
    case[-1].max_new = 0
    compare(case)


def test_many_groups():
    rng = random.Random(3)
    groups = [(rng.randrange(0, 4), [(rng.randrange(0, 40), rng.choice([0, 1, 1, 2])) for _ in range(rng.randrange(1, 5))])
              for _ in range(70)]
    compare(shared_case(groups, 8, 2, 64, 16, False, 10))
    compare(shared_case(groups, 16, 1, 64, 16, True, 11))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads,new", [(64, 24, 8, 1), (128, 24, 8, 1), (128, 40, 2, 2), (256, 24, 4, 3)])
def test_many_short_requests(dim, heads, kv_heads, new, q8):
    """Several row blocks in every range, most of them shorter than a tile."""
    rng = random.Random(dim + new)
    members = [(rng.choice([0, 1, 15, 16, 47, 48, 60, 63, 64, 65, 130]), rng.choice([0, new, new])) for _ in range(230)]
    compare(shared_case([(5, members), (0, members[:40]), (1, members[40:80])], heads, kv_heads, dim, 16, q8, 21))


@pytest.mark.parametrize("dim,heads", [(128, 6), (64, 3), (256, 4)])
def test_values_that_are_not_finite_among_drafted_tokens(dim, heads):
    """Infinities in keys' values that only some rows of a tile see, in pieces with and without
    them by turns, for row blocks behind one another in a range."""
    rng = random.Random(dim)
    members = [(rng.randrange(0, 50), rng.choice([1, 3])) for _ in range(200)]
    case = shared_case([(2, members)], heads * 4, 4, dim, 16, False, 22)
    cache, tables, lens, cu, q, step = case
    clean, _ = run(cache, q, step)
    want = clean.double().view(-1, heads * 4, dim).clone()
    for b in range(0, 200, 3):
        at = lens[b] + cu[b + 1] - cu[b] - 1  # the last new token: the earlier ones do not see it
        bad = float("inf") if b % 2 else float("-inf")
        cache.v[int(tables[b, at // 16]), b % 4, at % 16, b % dim] = bad
        want[cu[b + 1] - 1, b % 4 * heads:(b % 4 + 1) * heads, b % dim] = bad
    out, _ = run(cache, q, step)
    assert torch.equal(out.double().view(want.shape), want)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = random.Random(seed)
    kv_heads = rng.choice([1, 2, 4])
    heads = kv_heads * rng.choice([1, 2, 3, 6, 8, 12])
    page = rng.choice([16, 32, 48, 128])
    groups = []
    for _ in range(rng.randrange(1, 6)):
        members = [(None if rng.random() < 0.05 else rng.randrange(0, 300), rng.choice([0, 1, 1, 1, 2, 7]))
                   for _ in range(rng.choice([1, 2, 4, 9, 25]))]
        groups.append((rng.randrange(0, 3000 // page), members))
    if not any(n for _, m in groups for _, n in m):
        groups[0][1][0] = (4, 1)
    compare(shared_case(groups, heads, kv_heads, rng.choice([64, 128, 256]), page, rng.random() < 0.5, seed))


@pytest.mark.parametrize("what", ["not whole pages", "too long", "negative"])
def test_prefixes_that_do_not_fit_are_cut_and_reported(what):
    case = shared_case([(4, [(20, 1), (20, 1)])], 4, 2, 64, 16, False, 12)
    lens = {"not whole pages": [64 + 9] * 2, "too long": [1 << 20] * 2, "negative": [-5] * 2}[what]
    case[-1].prefix.lens = dev(lens, torch.int32)
    cache, tables, total, cu, q, step = case
    tables[1, :5] = tables[0, :5]  # 84 tokens: 80 of them in whole pages
    step.tables = dev(tables.tolist(), torch.int32)
    out = cache.attend(q.view(2, -1), step)
    if what == "negative":
        status()
    else:
        torch.cuda.synchronize()
        with pytest.raises(w12.W12Error) as e:
            w12.w12_check_status()
        assert e.value.status == 2
    want = attend_ref(q, cache, tables, total, cu, None, 0, 0.125, 2)
    check_attend(out, want[1], want)


@pytest.mark.parametrize("heads,q8", [(4, False), (40, False), (40, True), (32, True)])
@pytest.mark.parametrize("what", ["another length", "no group"])
def test_requests_that_do_not_fit_their_group(what, heads, q8):
    """They are reported and get zeros where they share another length; the others are right."""
    case = shared_case([(3, [(20, 1), (7, 1), (33, 1)]), (2, [(20, 1)] * 4)], heads, 2, 64, 16, q8, 23)
    cache, tables, total, cu, q, step = case
    if what == "another length":
        step.prefix.lens = dev([48, 32, 48, 32, 32, 32, 32], torch.int32)
        bad = [1]
    else:
        step.prefix.cu = dev([0, 3, 5], torch.int32)
        bad = [5, 6]  # what they get is not said
    lse = torch.zeros(7, heads, device="cuda")
    out = cache.attend(q.view(7, -1), step, lse=lse)
    torch.cuda.synchronize()
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 2
    want = attend_ref(q, cache, tables, total, cu, None, 0, 0.125, heads // 2)
    good = [b for b in range(7) if b not in bad]
    assert what == "no group" or (out[bad] == 0).all() and (lse[bad] == float("-inf")).all()
    check_attend(out[good], lse[good], tuple(w[good] for w in want))


def test_streams_graphs_and_workspaces():
    cache, tables, lens, cu, q, step = shared_case([(20, [(50, 1), (9, 1), (0, 1)])], 8, 2, 64, 16, False, 13)
    other = shared_case([(3, [(5, 2)] * 20)], 8, 2, 64, 16, False, 14)
    ref = attend_ref(q, cache, tables, lens, cu, None, 0, 0.125, 4)
    out, lse = torch.zeros(3, 512, device="cuda", dtype=torch.bfloat16), torch.zeros(3, 8, device="cuda")
    plain = KVStep(step.tables, step.lens, step.cu_new)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    cache.attend(q.view(3, -1), step, out=out, lse=lse, stream=stream)
    stream.synchronize()
    check_attend(out, lse, ref)
    graph = torch.cuda.CUDAGraph()
    cache.attend(q.view(3, -1), step)
    with torch.cuda.graph(graph, stream=stream):
        cache.attend(q.view(3, -1), step, out=out, lse=lse)
    for _ in range(3):
        out.zero_(), lse.zero_()
        graph.replay()
        y, z = run(cache, q, plain)  # the ordinary call, whose counters are its own
        torch.cuda.synchronize()
        check_attend(out, lse, ref)
        check_attend(y, z, ref)
        compare(other)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(w12.W12Error) as e:
        cache.attend(q.view(3, -1), step, workspace=small)
    assert e.value.status == 3
    mine = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")  # no initial contents are needed
    out, lse = run(cache, q, step, workspace=mine)
    check_attend(out, lse, ref)


def test_threads_on_one_stream():
    case = shared_case([(40, [(100, 1)] * 6)], 12, 2, 128, 16, False, 15)
    cache, tables, lens, cu, q, step = case
    want, _ = run(cache, q, step)
    got, errors = {}, []
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def work(i):
        try:
            for _ in range(50):
                got[i] = cache.attend(q.view(6, -1), step, stream=stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    stream.synchronize()
    assert not errors and all(torch.equal(y, want) for y in got.values())
    status()


def test_refusals():
    cache, _, _, _, q, step = shared_case([(2, [(5, 1), (9, 1)])], 4, 2, 64, 16, False, 16)
    with pytest.raises(w12.W12Error) as e:
        cache.attend(q.view(2, -1), step, window=5)
    assert e.value.status == 1
    step.prefix = KVPrefix(dev([0, 1, 1, 2], torch.int32), dev([0, 0], torch.int32))
    with pytest.raises(w12.W12Error) as e:  # more groups than requests
        cache.attend(q.view(2, -1), step)
    assert e.value.status == 2
    step.prefix = KVPrefix(dev([0, 2], torch.int32), dev([0, 0, 0], torch.int32))
    with pytest.raises(ValueError):
        cache.attend(q.view(2, -1), step)
    with pytest.raises(ValueError):
        KVPrefix(dev([0, 2], torch.int32), dev([0], torch.int64))
    with pytest.raises(ValueError):
        KVPrefix(torch.zeros(2, dtype=torch.int32), dev([0], torch.int32))
