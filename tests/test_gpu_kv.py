"""Paged key-value cache on the GPU: page planning, the store (norm, rotation,
cache write), reading back and attention, each against a plain 64-bit
implementation on the CPU."""
import math
import random

import numpy as np
import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVCache, KVPages, KVStep, w12

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def status():
    torch.cuda.synchronize()
    w12.w12_check_status()


def dev(x, dtype):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ---------------------------------------------------------------- plan
def plan_ref(lens, new, owned, tables, ring, state, page, blocks, tokens, trim):
    """The planning rules, one request at a time."""
    n = len(lens)
    tables, ring, (head, tail) = [list(r) for r in tables], list(ring), state
    src = list(ring)
    cap, avail = blocks * page, max(tail - head, 0)
    cu, pos, slots, owned_out = [0], [], [], []
    taken = back = 0
    for b in range(n):
        length = min(max(lens[b], 0), cap)
        add = min(max(new[b], 0), cap - length)
        have = min(max(owned[b], 0), blocks)
        need = -(-(length + add) // page)
        for j in range(have, need):
            tables[b][j] = src[(head + taken) % len(ring)] if taken < avail else -1
            have += taken < avail
            taken += 1
        if trim:
            for j in range(need, have):
                ring[(tail + back) % len(ring)] = tables[b][j]
                back += 1
            have = min(have, need)
        owned_out.append(have)
        for i in range(add):
            p = tables[b][(length + i) // page]
            pos.append(length + i)
            slots.append(-1 if p < 0 else p * page + (length + i) % page)
        cu.append(len(pos))
    pos, slots = pos[:tokens], slots[:tokens]
    pos += [0] * (tokens - len(pos))
    slots += [-1] * (tokens - len(slots))
    return tables, owned_out, ring, [head + min(taken, avail), tail + back], cu, pos, slots


def plan_case(n, kv, new, page, blocks, trim, seed, free=None):
    rng = random.Random(seed)
    lens = [rng.randint(0, kv) for _ in range(n)]
    add = [rng.randint(0, new) for _ in range(n)]
    owned = [min(blocks, -(-x // page) + (rng.randint(0, 3) if rng.random() < 0.3 else 0)) for x in lens]
    for b in range(n):
        if trim and rng.random() < 0.2:
            lens[b] = add[b] = 0
    total = sum(owned) + n * (-(-new // page) + 1)
    ids = list(range(total))
    rng.shuffle(ids)
    tables, at = [], 0
    for b in range(n):
        tables.append(ids[at:at + owned[b]] + [-1] * (blocks - owned[b]))
        at += owned[b]
    free = total - sum(owned) if free is None else min(free, total - sum(owned))
    head = rng.randrange(1 << 34)
    ring = [-7] * total
    for i in range(free):
        ring[(head + i) % total] = ids[at + i]
    return lens, add, owned, tables, ring, [head, head + free]


def run_plan(case, page, tokens, trim, in_place=True):
    lens, add, owned, tables, ring, state = case
    pages = KVPages(dev(tables, torch.int32), dev(owned, torch.int32), dev(ring, torch.int32),
                    dev(state, torch.int64), page)
    step = pages.step(tokens)
    out = {} if in_place else {"owned_out": torch.empty_like(pages.owned),
                               "ring_state_out": torch.empty_like(pages.ring_state)}
    pages.plan(dev(lens, torch.int32), dev(add, torch.int32), step, trim=trim, **out)
    torch.cuda.synchronize()
    if not in_place:
        assert pages.owned.tolist() == owned and pages.ring_state.tolist() == state
    return (pages.tables.tolist(), out.get("owned_out", pages.owned).tolist(), pages.ring.tolist(),
            out.get("ring_state_out", pages.ring_state).tolist(), step.cu_new.tolist(), step.positions.tolist(),
            step.slots.tolist())


@pytest.mark.parametrize("n,kv,new,page,blocks", [(1, 0, 1, 16, 4), (1, 500, 700, 16, 128), (7, 100, 33, 48, 9),
                                                  (256, 900, 1, 32, 40), (1024, 300, 9, 16, 24),
                                                  (1500, 200, 5, 64, 5), (2100, 60, 3, 16, 5)])
@pytest.mark.parametrize("trim", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
def test_plan(n, kv, new, page, blocks, trim, in_place):
    case = plan_case(n, kv, new, page, blocks, trim, seed=n + kv)
    tokens = n * new + 5
    got = run_plan(case, page, tokens, trim, in_place)
    want = plan_ref(*case, page, blocks, tokens, trim)
    for g, w, what in zip(got, want, ("tables", "owned", "ring", "ring_state", "cu_new", "positions", "slots")):
        assert g == w, what
    w12.w12_check_status()


def test_plan_ring_runs_out():
    case = plan_case(40, 100, 40, 16, 16, False, seed=5, free=21)
    got, want = run_plan(case, 16, 1700, False), plan_ref(*case, 16, 16, 1700, False)
    assert got == want
    assert -1 in got[6][:got[4][-1]]
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 3
    w12.w12_check_status()  # cleared


def test_plan_clamps_and_short_token_buffer():
    lens, add = [-3, 60, 10, 64], [4, 100, -2, 1]
    case = (lens, add, [0, 4, 1, 4], [[9] * 4] * 4, list(range(20)), [3, 15])
    got, want = run_plan(case, 16, 64, False), plan_ref(*case, 16, 4, 64, False)
    assert got == want and got[4] == [0, 4, 8, 8, 8]
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 2
    case = ([0, 0], [10, 10], [0, 0], [[-1] * 4] * 2, list(range(20)), [0, 20])
    got, want = run_plan(case, 16, 13, False), plan_ref(*case, 16, 4, 13, False)
    assert got == want
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 2


def test_plan_pages_given_back_are_taken_again():
    pages = KVPages.create(12, 16, requests=2, max_blocks=8)
    step = pages.step(256)
    lens = dev([0, 0], torch.int32)
    pages.plan(lens, dev([100, 60], torch.int32), step)
    assert pages.owned.tolist() == [7, 4]
    pages.plan(lens, dev([0, 60], torch.int32), step, trim=True)  # the first request is done
    assert pages.owned.tolist() == [0, 4] and pages.ring_state.tolist() == [11, 19]
    pages.plan(lens, dev([128, 60], torch.int32), step)
    assert pages.owned.tolist() == [8, 4]
    held = pages.tables.tolist()
    assert sorted(held[0] + held[1][:4]) == list(range(12))
    status()


# ---------------------------------------------------------------- store and read
def rope_table(rows, rot, seed=0):
    rng = np.random.default_rng(seed)
    a = rng.uniform(-math.pi, math.pi, (rows, rot // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def store_ref(x, weight, eps, rope, positions, interleaved):
    """(result, largest magnitude of the normed row) in 64 bits."""
    x = x.double().cpu()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    top = x.abs().amax(-1, keepdim=True)
    if rope is None:
        return x, top
    rot = rope.shape[1]
    row = rope.double().cpu()[positions.long().cpu()][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    y = x.clone()
    lo = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    hi = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y, top


def make_cache(pages, heads, page, dim, q8, layout="hnd", fill=None):
    shape = (pages, heads, page, dim) if layout == "hnd" else (pages, page, heads, dim)
    dtype = torch.int8 if q8 else torch.bfloat16
    mk = lambda: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    k, v = mk(), mk()
    if layout == "nhd":
        k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    if layout == "gap":  # pages and rows with room between them
        wide = torch.zeros(2, pages, heads, page + 2, dim + 16, dtype=dtype, device="cuda")
        k, v = wide[0, :, :, :page, :dim], wide[1, :, :, :page, :dim]
    scales = torch.zeros(pages, heads, page, 2, device="cuda") if q8 else None
    return KVCache(k, v, scales)


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 1), (128, 6, 2), (128, 48, 8), (256, 5, 5), (64, 3, 3)])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("tokens,rot,interleaved,norm,layout", [(1, "full", False, True, "hnd"),
                                                                (7, "half", False, True, "nhd"),
                                                                (33, "full", True, False, "gap"),
                                                                (130, 0, False, True, "hnd"),
                                                                (5, 6, True, True, "nhd"),
                                                                (2, 16, False, False, "hnd")])
def test_store_and_read(dim, heads, kv_heads, q8, tokens, rot, interleaved, norm, layout):
    g = torch.Generator(device="cuda").manual_seed(dim + tokens)
    rot = {"full": dim, "half": dim // 2}.get(rot, rot)
    page, pages = 16, tokens // 16 + 3
    cache = make_cache(pages, kv_heads, page, dim, q8, layout)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    # q, k and v as slices of one wide tensor: strides other than the heads' sum
    wide = 4 * rnd(tokens, (heads + 2 * kv_heads) * dim + 8)
    q = wide[:, :heads * dim]
    k = wide[:, heads * dim:(heads + kv_heads) * dim]
    v = wide[:, (heads + kv_heads) * dim:(heads + 2 * kv_heads) * dim]
    qw, kw = (rnd(dim), rnd(dim)) if norm else (None, None)
    rope = rope_table(50, rot) if rot else None
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:tokens]
    if tokens > 4:
        slots[3] = -1
    step = KVStep(positions=torch.randint(0, 50, (tokens,), device="cuda", generator=g, dtype=torch.int32), slots=slots)
    out = cache.store(q, k, v, step, q_norm=qw, k_norm=kw, eps=1e-5, rope=rope, interleaved=interleaved)
    got_k, got_v = cache.read(slots)
    status()
    ref, top = store_ref(q.reshape(tokens, heads, dim), qw, 1e-5, rope, step.positions, interleaved)
    # fp32 arithmetic (a few 2^-24 of the row's largest value) and one BF16 rounding (8 significant bits: 2^-8)
    assert ((out.view(tokens, heads, dim).double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * top).all()
    kref, ktop = store_ref(k.reshape(tokens, kv_heads, dim), kw, 1e-5, rope, step.positions, interleaved)
    vref = v.reshape(tokens, kv_heads, dim).double().cpu()
    here = (slots >= 0).cpu()
    for got, want, big in ((got_k, kref, ktop), (got_v, vref, vref.abs().amax(-1, keepdim=True))):
        got = got.double().cpu()
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -19 * big
        if q8:  # half a step of the row's scale, then the rounding of what read returns
            bound = bound + (0.501 * (1 + 2.0 ** -8)) * want.abs().amax(-1, keepdim=True) / 127
        assert ((got - want).abs() <= bound)[here].all()
        assert (got[~here] == 0).all()
    if not q8:
        assert torch.equal(got_v[here.cuda()], v.reshape(tokens, kv_heads, dim)[here.cuda()])
    # what read returns is what the cache holds
    at = slots.clamp(min=0)
    for i, (t, got) in enumerate(((cache.k, got_k), (cache.v, got_v))):
        held = t[at // page, :, at % page].float()
        if q8:
            held = held * cache.scales[at // page, :, at % page, i][..., None]
        assert torch.equal(held.to(torch.bfloat16)[here.cuda()], got[here.cuda()])
    # nothing else was written
    mask = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    mask[slots[slots >= 0]] = False
    for t in (cache.k, cache.v):
        assert (t.transpose(1, 2).reshape(pages * page, -1)[mask] == 0).all()


def test_store_in_place_and_without_q():
    cache = make_cache(2, 2, 16, 64, False)
    q = torch.randn(3, 4 * 64, device="cuda").to(torch.bfloat16)
    k, v = q[:, :128].clone(), q[:, 128:].clone()
    step = KVStep(positions=dev([1, 2, 3], torch.int32), slots=dev([5, 6, 31], torch.int64))
    rope = rope_table(4, 64)
    w = torch.randn(64, device="cuda").to(torch.bfloat16)
    want = cache.store(q, k, v, step, q_norm=w, rope=rope)  # a norm of q alone
    kept = cache.k.clone()
    got = cache.store(q, k, v, step, q_norm=w, rope=rope, out=q)
    assert got.data_ptr() == q.data_ptr() and got.shape == (3, 4, 64) and torch.equal(got, want)
    cache.k.zero_()
    assert cache.store(None, k, v, step, rope=rope) is None
    assert torch.equal(cache.k, kept)
    status()


def test_nothing_to_do():
    cache = make_cache(1, 2, 16, 64, False)
    none = torch.empty(0, 128, device="cuda", dtype=torch.bfloat16)
    step = KVStep(positions=dev([], torch.int32), slots=dev([], torch.int64))
    assert cache.store(none, none, none, step).shape == (0, 2, 64)
    a, b = cache.read(step.slots)
    assert a.shape == (0, 2, 64) and b.shape == (0, 2, 64)
    pages = KVPages.create(4, 16, requests=2, max_blocks=2)
    empty = pages.step(0)
    pages.plan(dev([0, 0], torch.int32), dev([0, 0], torch.int32), empty)
    assert empty.cu_new.tolist() == [0, 0, 0]
    status()


@pytest.mark.parametrize("q8", [False, True])
def test_store_zero_rows_and_values_that_are_not_finite(q8):
    cache = make_cache(1, 3, 16, 64, q8)
    k = torch.zeros(2, 3, 64, device="cuda", dtype=torch.bfloat16)
    k[0, 1, 7], k[0, 2, 9], k[1] = float("nan"), float("inf"), 1e-38
    step = KVStep(slots=dev([3, 4], torch.int64))
    cache.store(None, k, k, step)
    a, b = cache.read(step.slots)
    status()
    for t in (a, b):
        assert (t[0, 0] == 0).all()
        assert torch.isnan(t[0, 1, 7])
        if q8:  # the row's scale carries it
            assert torch.isnan(t[0, 1:]).all()
        else:
            assert torch.isinf(t[0, 2, 9]) and t[0, 1].isnan().sum() == 1
        assert ((t[1].float() - 1e-38).abs() <= 1e-40).all()


def test_store_and_read_report_bad_indices():
    for slots, positions in (([0, 32], [0, 0]), ([0, 1], [0, 9]), ([0, 1], [-1, 0])):
        cache = make_cache(2, 1, 16, 64, False)
        k = torch.ones(2, 64, device="cuda", dtype=torch.bfloat16)
        step = KVStep(positions=dev(positions, torch.int32), slots=dev(slots, torch.int64))
        cache.store(None, k, k, step, rope=rope_table(9, 64))
        with pytest.raises(w12.W12Error) as e:
            w12.w12_check_status()
        assert e.value.status == 1
    cache = make_cache(2, 1, 16, 64, True)
    a, _ = cache.read(dev([99], torch.int64))
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 1 and (a == 0).all()


# ---------------------------------------------------------------- attend
def held_rows(cache, table, count):
    """Keys and values of a request's first `count` tokens in 64 bits, and which are present."""
    page, n = cache.page_size, cache.k.shape[0]
    j = np.arange(count)
    p = table[j // page] if count else np.zeros(0, int)
    ok = torch.from_numpy((p >= 0) & (p < n))
    p, off = torch.from_numpy(np.clip(p, 0, n - 1)).cuda(), torch.from_numpy(j % page).cuda()
    out = []
    for i, t in enumerate((cache.k, cache.v)):
        x = t[p, :, off].double()
        if cache.scales is not None:
            x = x * cache.scales[p, :, off, i].double()[..., None]
        out.append(x.cpu())
    return out[0], out[1], ok


def attend_ref(q, cache, tables, lens, cu, tree, window, scale, group):
    """(out, lse, sum of weight * |v|, largest sum of |q k| * scale) in 64 bits."""
    t, h = q.shape[0], q.shape[1]
    out = torch.zeros(t, h, q.shape[2], dtype=torch.float64)
    mass, lse, big = out.clone(), torch.full((t, h), -math.inf, dtype=torch.float64), torch.zeros(t, h, dtype=torch.float64)
    q = q.double().cpu()
    for b, past in enumerate(lens):
        m = cu[b + 1] - cu[b]
        k, v, ok = held_rows(cache, tables[b], past + m)
        key = torch.arange(past + m)
        for i in range(m):
            see = ok & (key <= past + i)
            if tree is not None:
                bits = int(tree[cu[b] + i]) & 0xFFFFFFFF
                see = ok & ((key < past) | torch.tensor([j >= past and j - past < 32 and bits >> (j - past) & 1 == 1
                                                         for j in range(past + m)], dtype=torch.bool))
            if window:
                see &= key > past + i - window
            if not see.any():
                continue
            kk, vv = (x[see].repeat_interleave(group, 1) for x in (k, v))
            row = q[cu[b] + i]
            s = torch.einsum("hd,khd->hk", row, kk) * scale
            w = torch.softmax(s, -1)
            out[cu[b] + i] = torch.einsum("hk,khd->hd", w, vv)
            mass[cu[b] + i] = torch.einsum("hk,khd->hd", w, vv.abs())
            lse[cu[b] + i] = torch.logsumexp(s, -1)
            big[cu[b] + i] = (torch.einsum("hd,khd->hk", row.abs(), kk.abs()) * abs(scale)).amax(-1)
    return out, lse, mass, big


def check_attend(out, lse, ref, what=""):
    want, want_lse, mass, big = ref
    out, lse = out.double().cpu().view(want.shape), lse.double().cpu()
    # BF16 weights: 2^-8 of each; fp32 scores: see lse; BF16 output: 2^-8
    bound = 2.0 ** -8 * want.abs() + (1.1 * 2.0 ** -8 + 2.0 ** -17 * big[..., None]) * mass
    bad = ~((out - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(out - want).abs()[bad].max()}"
    # at most 2^-22 per 16-column step of the sum, and the exponential's and logarithm's own
    none = torch.isinf(want_lse)
    assert torch.equal(none, torch.isinf(lse)) and (lse[none] < 0).all()
    assert ((lse - want_lse).abs()[~none] <= (1e-5 * (1 + want_lse.abs()) + 2.0 ** -18 * big)[~none]).all(), what


def attend_case(lens, new, heads, kv_heads, dim, page, q8, seed, layout="hnd", spare=2, stale=True):
    """A cache with the requests' pages in random places, stale memory behind
    each request's last token, and the step."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-(a + b) // page) for a, b in zip(lens, new)]
    pages = sum(need) + spare
    cache = make_cache(pages, kv_heads, page, dim, q8, layout)
    if q8:
        for t in (cache.k, cache.v):
            t.copy_(torch.randint(-127, 128, t.shape, device="cuda", generator=g, dtype=torch.int8))
        cache.scales.copy_(torch.rand(cache.scales.shape, device="cuda", generator=g) * 0.01 + 0.005)
    else:
        for t in (cache.k, cache.v):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
    ids = rng.permutation(pages)
    width = max(need + [1]) + 1
    tables = np.full((len(lens), width), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
        left = lens[b] + new[b] - (n - 1) * page
        if stale and n and left < page:
            last = int(tables[b, n - 1])
            for t in (cache.scales,) if q8 else (cache.k, cache.v):
                t[last, :, left:] = float("nan")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    step = KVStep(dev(tables.tolist(), torch.int32), dev(lens, torch.int32), dev(cu, torch.int32), max_new=max(new + [1]))
    return cache, tables, cu, q, step


def run_attend(cache, q, step, **kw):
    t, h, d = q.shape
    lse = torch.full((t, h), 7.0, device="cuda")
    out = cache.attend(q.reshape(t, h * d), step, lse=lse, **kw)
    status()
    return out, lse


HEADS = [(64, 8, 8), (64, 8, 1), (128, 12, 2), (128, 5, 1), (256, 6, 1), (256, 4, 2), (128, 33, 1), (64, 20, 1)]


@pytest.mark.parametrize("dim,heads,kv_heads", HEADS)
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,new,page", [([0], [1], 16), ([15], [1], 16), ([63, 64, 65, 0, 200], [1, 1, 1, 1, 1], 32),
                                           ([1000], [1], 48), ([5, 0, 130, 77], [3, 0, 8, 1], 16),
                                           ([0, 300], [20, 17], 64)])
def test_attend(dim, heads, kv_heads, q8, lens, new, page):
    cache, tables, cu, q, step = attend_case(lens, new, heads, kv_heads, dim, page, q8, seed=dim + heads + len(lens))
    out, lse = run_attend(cache, q, step)
    ref = attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, heads // kv_heads)
    check_attend(out, lse, ref)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("window", [1, 16, 63, 64, 100, 5000])
@pytest.mark.parametrize("group,dim", [(3, 128), (11, 128), (17, 64), (9, 256)])
def test_attend_window(q8, window, group, dim):
    lens, new = [0, 300, 64, 127], [2, 5, 1, 1]
    cache, tables, cu, q, step = attend_case(lens, new, 2 * group, 2, dim, 16, q8, seed=window)
    out, lse = run_attend(cache, q, step, window=window, scale=0.2)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, window, 0.2, group))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 4), (128, 12, 2), (256, 6, 1)])
@pytest.mark.parametrize("window", [0, 40])
def test_attend_tree(q8, dim, heads, kv_heads, window):
    lens, new = [0, 100, 48, 7], [6, 16, 32, 1]
    cache, tables, cu, q, step = attend_case(lens, new, heads, kv_heads, dim, 16, q8, seed=dim + heads)
    rng = random.Random(dim)
    masks = []
    for n in new:
        m = []
        for i in range(n):
            m.append((m[rng.randrange(i)] if i else 0) | 1 << i)
        masks += m
    masks[0] = 0          # with nothing cached: a row that sees nothing
    masks[2] = 1 << 5     # a later token, and not itself
    masks[9] = 0xFFFFFFFF  # bits behind the request's last token
    tree = np.array(masks, np.uint32).view(np.int32)
    step.tree = torch.from_numpy(tree).cuda()
    out, lse = run_attend(cache, q, step, window=window)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, tree, window, dim ** -0.5, heads // kv_heads))
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()


@pytest.mark.parametrize("layout", ["nhd", "gap"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_layouts_and_strided_q(layout, q8, dim):
    lens, new = [70, 3], [1, 2]
    cache, tables, cu, q, step = attend_case(lens, new, 4, 2, dim, 16, q8, seed=3, layout=layout)
    wide = torch.zeros(3, 6 * dim, device="cuda", dtype=torch.bfloat16)
    wide[:, dim:5 * dim] = q.view(3, -1)
    out = torch.full((3, 7 * dim), 9.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(3, 4, device="cuda")
    cache.attend(wide[:, dim:5 * dim], step, out=out[:, 2 * dim:6 * dim], lse=lse)
    status()
    check_attend(out[:, 2 * dim:6 * dim].reshape(3, -1), lse, attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, 2))
    assert (out[:, :2 * dim] == 9).all() and (out[:, 6 * dim:] == 9).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 2, 1], [16, 7, 25]])
def test_attend_long_split_over_ctas(q8, dim, new):
    """One request over many CTAs, beside short ones; the same bits every time."""
    lens = [9000, 3, 700]
    cache, tables, cu, q, step = attend_case(lens, new, 6, 1, dim, 16, q8, seed=dim)
    out, lse = run_attend(cache, q, step)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, 6))
    for _ in range(3):
        again, lse2 = run_attend(cache, q, step)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [2, 40])
@pytest.mark.parametrize("q8", [False, True])
def test_attend_absent_pages(group, q8, dim):
    lens, new = [200, 40], [1, 1]
    cache, tables, cu, q, step = attend_case(lens, new, 2 * group, 2, dim, 16, q8, seed=8)
    tables[0, 2], tables[0, 4], tables[0, 8:12], tables[1, :] = -1, 1 << 20, -1, -5
    step.tables.copy_(torch.from_numpy(tables))
    out, lse = run_attend(cache, q, step)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, group))
    assert (out[1] == 0).all() and torch.isinf(lse[1]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("group", [3, 12])  # the warp-level and the tcgen05 kernel
def test_attend_unseen_values_have_no_effect(dim, bad, q8, group):
    """Drafted tokens whose keys and values are not finite: the tokens that do
    not see them are as if they were not there; those that do are not finite."""
    lens, new = [37], [5]
    cache, tables, cu, q, step = attend_case(lens, new, 2 * group, 2, dim, 16, q8, seed=1)
    tree = np.array([1, 2, 5, 10, 0b10001], np.int32)  # token 1 is seen by 1 and 3 alone
    step.tree = torch.from_numpy(tree).cuda()
    ref = attend_ref(q, cache, tables, lens, cu, tree, 0, dim ** -0.5, group)
    page, off = int(tables[0, 38 // 16]), 38 % 16
    if q8:
        cache.scales[page, 1, off] = bad
    else:
        cache.v[page, 1, off, 3:9] = bad
        cache.k[page, 1, off, 2] = bad
    out, lse = run_attend(cache, q, step)
    clean = [0, 2, 4]
    check_attend(out[clean], lse[clean], tuple(x[clean] for x in ref))
    out = out.view(5, 2 * group, dim)
    check_attend(out[:, :group], lse[:, :group], tuple(x[:, :group] for x in ref))
    if bad != bad:
        assert torch.isnan(out[1, group:, 3:9]).all() and torch.isnan(out[3, group:, 3:9]).all()
    # a request behind it is not touched by what this one met
    again, lse2 = run_attend(cache, q, step)
    assert torch.equal(again.view(out.shape)[clean], out[clean]) and torch.equal(lse2[clean], lse[clean])


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (40, 2, 64), (40, 2, 128), (20, 1, 256)])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_attend_large_scores(heads, kv_heads, dim, scale):
    """Scores far apart and far from zero: the running maximum is raised again and again."""
    lens, new = [400], [2]
    cache, tables, cu, q, step = attend_case(lens, new, heads, kv_heads, dim, 16, False, seed=4)
    cache.k.mul_(torch.linspace(-30, 60, cache.k.shape[0], device="cuda")[:, None, None, None])
    out, lse = run_attend(cache, q, step, scale=scale)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, 0, scale, heads // kv_heads))


def test_attend_rows_without_tokens_and_more_rows_than_max_new_says():
    lens, new = [50, 9], [9, 4]
    cache, tables, cu, q, step = attend_case(lens, new, 6, 2, 128, 16, False, seed=5)
    step.max_new = 1  # a wrong bound only picks another tile
    q2 = torch.cat([q, torch.full_like(q[:2], float("nan"))])
    out = torch.full((15, 6 * 128), 3.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((15, 6), 3.0, device="cuda")
    cache.attend(q2.view(15, -1), step, out=out, lse=lse)
    status()
    check_attend(out[:13], lse[:13], attend_ref(q, cache, tables, lens, cu, None, 0, 128 ** -0.5, 3))
    assert (out[13:] == 3).all() and (lse[13:] == 3).all()


@pytest.mark.parametrize("most,heads,kv_heads", [(2, 4, 2), (30, 8, 2)])
@pytest.mark.parametrize("q8", [False, True])
def test_attend_many_requests(most, heads, kv_heads, q8):
    rng = random.Random(0)
    lens = [rng.randint(0, 90) for _ in range(300)]
    new = [rng.choice([0, 1, 1, most]) for _ in range(300)]
    cache, tables, cu, q, step = attend_case(lens, new, heads, kv_heads, 64, 16, q8, seed=6)
    out, lse = run_attend(cache, q, step)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, 0, 0.125, heads // kv_heads))


@pytest.mark.parametrize("seed", range(40))
def test_attend_random_shapes(seed):
    rng = random.Random(seed)
    dim, kv_heads, group = rng.choice([64, 128, 256]), rng.choice([1, 2, 3]), rng.choice([1, 2, 5, 6, 16, 33])
    n, page, q8 = rng.randint(1, 40), rng.choice([16, 32, 48, 80, 128]), rng.random() < 0.5
    most = rng.choice([1, 1, 2, 3, 7, 20])
    lens = [rng.choice([0, rng.randint(0, 40), rng.randint(0, 700), rng.randint(60, 70)]) for _ in range(n)]
    new = [rng.choice([most, most, rng.randint(0, most)]) for _ in range(n)]
    if not sum(new):
        new[0] = 1
    window = rng.choice([0, 0, rng.randint(1, 200)])
    cache, tables, cu, q, step = attend_case(lens, new, kv_heads * group, kv_heads, dim, page, q8, seed)
    tree = None
    if most > 1 and rng.random() < 0.5:
        tree = np.array([rng.getrandbits(32) for _ in range(cu[-1])], np.uint32).view(np.int32)
        step.tree = torch.from_numpy(tree).cuda()
    out, lse = run_attend(cache, q, step, window=window)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, tree, window, dim ** -0.5, group))


def test_attend_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^32."""
    page, heads, dim = 16, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 40
    cache = KVCache.empty(pages, page, heads, dim)
    lens, new = [40], [1]
    tables = np.array([[pages - 1, 2, pages - 33, -1]])
    for p in (pages - 1, 2, pages - 33):
        cache.k[p] = torch.randn(heads, page, dim, device="cuda").to(torch.bfloat16)
    step = KVStep(dev(tables.tolist(), torch.int32), dev(lens, torch.int32), dev([0, 1], torch.int32),
                  slots=dev([(pages - 33) * page + 8], torch.int64))
    q, k, v = (torch.randn(1, heads, dim, device="cuda").to(torch.bfloat16) for _ in range(3))
    for p in (pages - 1, 2, pages - 33):
        cache.v[p] = torch.randn(heads, page, dim, device="cuda").to(torch.bfloat16)
    cache.store(None, k, v, step)
    got_k, got_v = cache.read(step.slots)
    out, lse = run_attend(cache, q, step)
    assert torch.equal(got_k, k) and torch.equal(got_v, v)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, [0, 1], None, 0, dim ** -0.5, 1))


def test_other_streams_and_graph():
    """A whole step on a side stream, captured in a graph and replayed on new lengths."""
    heads, kv_heads, dim, page = 6, 2, 128, 16
    pages = KVPages.create(64, page, requests=3, max_blocks=16)
    cache = make_cache(64, kv_heads, page, dim, False)
    step = pages.step(3)
    lens, new = dev([0, 0, 0], torch.int32), dev([1, 1, 1], torch.int32)
    rnd = lambda h: torch.zeros(3, h * dim, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, rope = rnd(heads), rnd(kv_heads), rnd(kv_heads), rope_table(256, dim)
    out, lse = torch.empty_like(q), torch.empty(3, heads, device="cuda")
    side = torch.cuda.Stream()

    def call():
        pages.plan(lens, new, step, stream=side)
        cache.store(q, k, v, step, rope=rope, out=q, stream=side)
        cache.attend(q, step, out=out, lse=lse, stream=side)

    torch.cuda.synchronize()
    call()
    side.synchronize()
    w12.w12_check_status(side)
    lens.fill_(1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    history = []
    g = torch.Generator(device="cuda").manual_seed(0)
    for t in range(1, 40):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        w12.w12_check_status()
        lens.add_(1)
        history.append(None)
    lens.sub_(1)
    ref = attend_ref(q.view(3, heads, dim), cache, pages.tables.cpu().numpy().astype(np.int64), lens.tolist(),
                     [0, 1, 2, 3], None, 0, dim ** -0.5, 3)
    check_attend(out, lse, ref)
    assert step.positions.tolist() == [39, 39, 39] and pages.owned.tolist() == [3, 3, 3]


def test_workspace_shared_by_calls_of_other_shapes():
    """One workspace for calls whose plans differ: each leaves its counters zero for the others."""
    cases = [attend_case([700, 20], [1, 1], 6, 1, 128, 16, False, seed=1),
             attend_case([100] * 50, [2] * 50, 8, 4, 64, 16, True, seed=2),
             attend_case([2000], [16], 6, 1, 256, 16, False, seed=3)]
    refs = [attend_ref(q, c, t, s.lens.tolist(), cu, None, 0, q.shape[2] ** -0.5, q.shape[1] // c.kv_heads)
            for c, t, cu, q, s in cases]
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for (c, t, cu, q, s), ref in zip(cases, refs):
            out, lse = run_attend(c, q, s, workspace=ws)
            check_attend(out, lse, ref)


def test_holders_refuse():
    cache = make_cache(2, 2, 16, 64, False)
    step = KVStep(dev([[0, 1]], torch.int32), dev([3], torch.int32), dev([0, 1], torch.int32),
                  positions=dev([3], torch.int32), slots=dev([3], torch.int64))
    q = torch.zeros(1, 4 * 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(1, 2 * 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cache.attend(q.float(), step)
    with pytest.raises(ValueError):
        cache.attend(q[:, :100], step)
    with pytest.raises(w12.W12Error) as e:
        cache.attend(q[:, :64], step)  # one head for two key heads
    assert e.value.status == 2
    with pytest.raises(w12.W12Error) as e:
        cache.attend(q, step, window=-1)
    assert e.value.status == 1
    with pytest.raises(w12.W12Error) as e:
        cache.attend(q, step, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(ValueError):
        cache.attend(q, step, lse=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        cache.store(q, kv[:, :64], kv, step)
    with pytest.raises(ValueError):
        cache.store(q, kv, kv, step, q_norm=torch.zeros(32, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(w12.W12Error) as e:
        cache.store(q, kv, kv, step, rope=torch.zeros(4, 24, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(ValueError):
        cache.read(dev([1], torch.int32))
    with pytest.raises(ValueError):
        KVCache(cache.k, cache.v.to(torch.int8))
    with pytest.raises(ValueError):
        KVCache(cache.k.to(torch.int8), cache.v.to(torch.int8))
    with pytest.raises(ValueError):
        KVPages(step.tables, step.lens, dev([1], torch.int64), dev([0, 1], torch.int64), 16)
    assert cache.attend(q[:0], step).shape == (0, 256)
    status()


@pytest.mark.parametrize("heads,kv_heads,dim", [(24, 2, 64), (40, 2, 128), (40, 2, 256), (6, 2, 128)])
def test_attend_infinite_values_among_many_short_requests(heads, kv_heads, dim):
    # several short requests per CTA, every other one with infinities that its row sees
    lens = [(37 * b) % 150 for b in range(331)]
    cache, tables, cu, q, step = attend_case(lens, [1] * len(lens), heads, kv_heads, dim, 16, False, 21)
    hit = torch.zeros(len(lens), kv_heads, dim, dtype=torch.bool)
    for b in range(0, len(lens), 2):
        for head, col in ((b % kv_heads, b % dim), (0, dim - 1)):
            key = lens[b] - (b % 3 if lens[b] > 2 else 0)
            cache.v[int(tables[b, key // 16]), head, key % 16, col] = math.inf
            hit[b, head, col] = True
    out, lse = run_attend(cache, q, step)
    hit = hit.repeat_interleave(heads // kv_heads, 1)
    out = out.view(hit.shape).cpu()
    assert (out[hit] == math.inf).all() and torch.isfinite(out[~hit]).all()
    ref = attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, heads // kv_heads)
    for x in (out, ref[0], ref[2]):
        x.masked_fill_(hit, 0.0)
    check_attend(out, lse, ref)


def test_workspace_outgrown_after_a_capture():
    # 2^18 + 64 row blocks need more counters than the first MiB of them holds
    cache, tables, cu, q, step = attend_case([700, 20], [1, 1], 4, 1, 64, 16, False, 22)
    ref = attend_ref(q, cache, tables, [700, 20], cu, None, 0, 0.125, 4)
    stream = torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    with torch.cuda.stream(stream):
        cache.attend(q, step, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        cache.attend(q, step, out=out, lse=lse)
    n = (1 << 18) + 64
    many = KVStep(step.tables[:1].expand(n, -1).contiguous(), torch.zeros(n, dtype=torch.int32, device="cuda"),
                  torch.arange(n + 1, dtype=torch.int32, device="cuda"))
    with torch.cuda.stream(stream):
        big = cache.attend(q[:1].expand(n, -1, -1).contiguous(), many)
    fill = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")  # whatever memory was given back
    out.zero_(), lse.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check_attend(out, lse, ref)
    # one visible key: its value (BF16) is the output
    first = cache.v[int(tables[0, 0]), 0, 0]
    assert (big.view(n, 4, 64) == first).all()
    del fill
    status()


def test_calls_refuse_what_is_no_tensor_or_does_not_fit():
    cache = make_cache(2, 2, 16, 64, False)
    step = KVStep(dev([[0, 1]], torch.int32), dev([3], torch.int32), dev([0, 1], torch.int32),
                  positions=dev([3], torch.int32), slots=dev([3], torch.int64))
    q = torch.zeros(1, 4 * 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(1, 2 * 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cache.attend([1.0], step)
    with pytest.raises(TypeError):
        cache.store(q, None, kv, step)
    with pytest.raises(TypeError):
        cache.read(3)
    with pytest.raises(ValueError):
        cache.attend(q, step, window=1 << 32)
    with pytest.raises(ValueError):
        cache.attend(q.cpu(), step)
    with pytest.raises(ValueError):
        cache.store(q, kv.cpu(), kv, step)
    with pytest.raises(TypeError):
        cache.attend(q, KVStep(step.tables, None, step.cu_new))
    with pytest.raises(ValueError):
        cache.read(step.slots, out=(kv.view(1, 2, 64), kv.float().view(1, 2, 64)))
    with pytest.raises(TypeError):
        KVPages(step.tables, step.lens, dev([1], torch.int32), dev([0, 1], torch.int64), 16).plan(
            step.lens, [1], step)


def test_store_returns_out_by_heads():
    cache = make_cache(2, 2, 16, 64, False)
    step = KVStep(slots=dev([0, 17, -1], torch.int64))
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = (torch.randn(3, n * 64, device="cuda", generator=g).to(torch.bfloat16) for n in (4, 2))
    wide = torch.zeros(3, 304, device="cuda", dtype=torch.bfloat16)
    out = wide[:, 24:280]
    y = cache.store(q, k, k, step, out=out)
    assert y.shape == (3, 4, 64) and y.data_ptr() == out.data_ptr() and y.stride() == (304, 64, 1)
    assert torch.equal(y.reshape(3, 256), q) and torch.equal(out, q)
    y.mul_(2)
    assert torch.equal(out, 2 * q) and not wide[:, :24].any() and not wide[:, 280:].any()
    three = torch.empty(3, 4, 64, device="cuda", dtype=torch.bfloat16)
    assert cache.store(q, k, k, step, out=three) is three
    fresh = cache.store(q, k, k, step)
    assert fresh.shape == (3, 4, 64) and torch.equal(fresh.view(3, 256), q)


def test_calls_by_the_c_names():
    # pages, store, read and attention by raw pointers, as the holders make them
    pages = KVPages.create(6, 16, 2, 4)
    cache = make_cache(6, 2, 16, 64, False)
    lens, new = dev([0, 0], torch.int32), dev([20, 9], torch.int32)
    step = pages.step(29, max_new=20)
    n, t = 2, 29
    w12.w12_kv_plan(w12.w12_kv_plan_args(
        lens.data_ptr(), new.data_ptr(), pages.owned.data_ptr(), pages.owned.data_ptr(), pages.tables.data_ptr(), 4,
        pages.ring.data_ptr(), pages.ring_state.data_ptr(), pages.ring_state.data_ptr(), step.cu_new.data_ptr(),
        step.positions.data_ptr(), step.slots.data_ptr(), n, 4, 16, 6, t, 0))
    assert pages.owned.tolist() == [2, 1] and step.cu_new.tolist() == [0, 20, 29]
    step.lens = lens
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(t, h * 64, device="cuda", generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    c, out = cache._c, torch.empty_like(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    w12.w12_kv_store(c, w12.w12_kv_store_args(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), 256, 128, 128, 256, None, None, None, None,
        step.slots.data_ptr(), 0, t, 4, 0, 0, 1e-6), stream)
    kk, vv = (torch.empty(t, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w12.w12_kv_read(c, step.slots.data_ptr(), t, kk.data_ptr(), vv.data_ptr(), stream)
    args = w12.w12_kv_attend_args(out.data_ptr(), out.data_ptr(), None, 256, 256, step.tables.data_ptr(), 4,
                                  lens.data_ptr(), step.cu_new.data_ptr(), None, n, 4, t, 4, 20, 0, 0.125)
    y = torch.empty_like(q)
    args.out = y.data_ptr()
    ws = torch.zeros(w12.w12_kv_attend_workspace_size(c, args), dtype=torch.uint8, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    w12.w12_kv_attend(c, args, ws.data_ptr(), ws.numel(), stream)
    torch.cuda.synchronize()
    status()
    assert torch.equal(out, q) and torch.equal(kk.view(t, -1), k) and torch.equal(vv.view(t, -1), v)
    assert torch.equal(y, cache.attend(out, step))
