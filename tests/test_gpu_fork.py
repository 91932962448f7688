"""Pages that requests share on the GPU: forking, taking back, freeing, the copies that come
out of it and the common prefix, against the rules applied one row at a time."""
import random

import pytest
import torch
from test_gpu_kv import dev, make_cache, status

from lossless_bit_weight_encode_gb300 import KVCopies, KVPages, KVPrefix, w12

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


class Pool:
    """The state of KVPages on the host, and the rules of fork."""

    def __init__(self, tables, owned, ring, state, shares, page):
        self.tables, self.owned, self.ring = [list(r) for r in tables], list(owned), list(ring)
        self.head, self.tail = state
        self.shares, self.page = list(shares), page

    def fork(self, parents, lens, groups=None):
        n, page = len(parents), self.page
        count = len(self.shares)
        old, owned = [list(r) for r in self.tables], list(self.owned)
        page_of = lambda r, c: old[r][c] if 0 <= old[r][c] < count else -1  # noqa: E731
        keep, need = [], []
        for i in range(n):
            real = 0 <= parents[i] < n
            keep.append(min(max(lens[i], 0), owned[parents[i]] * page) if real else 0)
            need.append(-(-keep[i] // page))
        holders = {}
        add = lambda p, k: holders.__setitem__(p, holders.get(p, self.shares[p] + 1) + k)  # noqa: E731
        for r in range(n):
            for c in range(owned[r]):
                if page_of(r, c) >= 0:
                    add(page_of(r, c), -1)
        for i in range(n):
            for c in range(keep[i] // page):
                if page_of(parents[i], c) >= 0:
                    add(page_of(parents[i], c), 1)
        src, dst, rows, taken = [-1] * n, [-1] * n, [0] * n, 0
        avail = self.tail - self.head
        new = [list(r) for r in self.tables]
        ring = list(self.ring)
        for i in range(n):
            for c in range(keep[i] // page):
                new[i][c] = page_of(parents[i], c)
            if keep[i] % page == 0:
                continue
            p = page_of(parents[i], need[i] - 1)
            new[i][need[i] - 1] = p
            if p < 0:
                continue
            if holders[p] == 0:
                holders[p] = 1  # the first that wants it keeps it
                continue
            new[i][need[i] - 1] = -1
            if taken < avail:
                q = self.ring[(self.head + taken) % len(ring)]
                new[i][need[i] - 1], src[i], dst[i], rows[i] = q, p, q, keep[i] % page
            taken += 1
        freed = []
        for c in range(max(owned + [0])):
            for r in range(n):
                p = page_of(r, c) if c < owned[r] else -1
                if p >= 0 and holders[p] == 0:
                    holders[p] = 1  # once
                    freed.append(p)
        for k, p in enumerate(freed):
            ring[(self.tail + k) % len(ring)] = p
        for p, h in holders.items():
            self.shares[p] = h - 1
        self.tables, self.owned, self.ring = new, need, ring
        self.head, self.tail = self.head + min(taken, avail), self.tail + len(freed)
        prefix = None
        if groups:
            prefix = [0] * n
            for a, b in zip(groups, groups[1:]):
                live = [i for i in range(a, b) if keep[i] > 0]
                if len(live) < 2:
                    continue
                same = 0
                while all(same < keep[i] // page and new[i][same] >= 0 and new[i][same] == new[live[0]][same]
                          for i in live):
                    same += 1
                for i in live:
                    prefix[i] = same * page
        return keep, src, dst, rows, prefix


def holders_of(pages, free_from=0):
    """Every page is in the ring or held, and shares says by how many."""
    count = {}
    tables, owned = pages.tables.tolist(), pages.owned.tolist()
    for r, n in enumerate(owned):
        for p in tables[r][:n]:
            count[p] = count.get(p, 0) + 1
    head, tail = pages.ring_state.tolist()
    ring = pages.ring.tolist()
    free = [ring[i % len(ring)] for i in range(head, tail)]
    assert len(set(free)) == len(free) and not set(free) & set(count)
    shares = pages.shares.tolist()
    assert sorted(free + list(count)) == list(range(len(shares)))
    assert all(shares[p] == count.get(p, 1) - 1 for p in range(len(shares)))


def case(rows, blocks, page, beams, seed, extra=0):
    """Rows in groups of `beams` that share a number of pages, in the state and on the host."""
    rng = random.Random(seed)
    count = rows * (blocks + 1) + extra
    ids = list(range(count))
    rng.shuffle(ids)
    tables, owned, shares, lens = [], [], [0] * count, []
    while len(tables) < rows:
        n = min(beams, rows - len(tables))
        total = rng.randint(1, blocks * page)
        held = -(-total // page)
        common = rng.randint(0, total // page)
        first = [ids.pop() for _ in range(common)]
        for p in first:
            shares[p] = n - 1
        for _ in range(n):
            more = min(blocks, held + rng.choice([0, 0, 0, 1, 2]))  # pages of drafted tokens
            tables.append(first + [ids.pop() for _ in range(more - common)] + [-1] * (blocks - more))
            owned.append(more)
            lens.append(total)
    head = rng.randrange(1000)
    ring = [-1] * count
    for i, p in enumerate(ids):
        ring[(head + i) % count] = p
    state = (head, head + len(ids))
    pages = KVPages(dev(tables, torch.int32), dev(owned, torch.int32), dev(ring, torch.int32),
                    dev(list(state), torch.int64), page, shares=dev(shares, torch.int32))
    return pages, Pool(tables, owned, ring, state, shares, page), lens


def run(pages, pool, parents, lens, groups=None, lens_out=True):
    n = len(parents)
    want = pool.fork(parents, lens, groups)
    prefix = KVPrefix(dev(groups, torch.int32), dev([7] * n, torch.int32)) if groups else None
    at = dev(lens, torch.int32)
    copies = pages.fork(dev(parents, torch.int32), at, prefix=prefix, lens_out=at if lens_out else None)
    torch.cuda.synchronize()
    keep, src, dst, rows, common = want
    assert pages.tables.tolist() == pool.tables and pages.owned.tolist() == pool.owned
    assert pages.ring.tolist() == pool.ring and pages.ring_state.tolist() == [pool.head, pool.tail]
    assert pages.shares.tolist() == pool.shares
    assert copies.src.tolist() == src and copies.dst.tolist() == dst and copies.rows.tolist() == rows
    assert at.tolist() == (keep if lens_out else lens)
    if groups:
        assert prefix.lens.tolist() == common
    return copies


@pytest.mark.parametrize("rows,blocks,page,beams", [(1, 1, 16, 1), (4, 7, 16, 4), (4, 64, 16, 4), (5, 9, 48, 2),
                                                    (33, 20, 32, 8), (96, 130, 16, 16), (130, 8, 64, 7),
                                                    (600, 33, 16, 5), (1024, 24, 16, 8), (4096, 3, 16, 32)])
@pytest.mark.parametrize("seed", [0, 1])
def test_fork(rows, blocks, page, beams, seed):
    pages, pool, lens = case(rows, blocks, page, beams, seed)
    rng = random.Random(100 + seed)
    groups = list(range(0, rows, beams)) + [rows]
    for step in range(3):
        parents, want = [], []
        for a, b in zip(groups, groups[1:]):
            done = rng.random() < 0.1
            back = rng.choice([0, 0, 1, page, 3 * page + 1])
            for i in range(a, b):
                p = -1 if done or rng.random() < 0.1 else rng.randrange(a, b)
                parents.append(p)
                want.append(max(0, min(lens[p], pool.owned[p] * page) - back) if p >= 0 else rng.choice([0, 5]))
        run(pages, pool, parents, want, groups if step != 1 else None, lens_out=step != 2)
        status()
        holders_of(pages)
        lens = [max(0, min(w, o * page)) for w, o in zip(want, pool.owned)]


def test_rows_of_any_other_and_different_lengths():
    # rows that go on from rows of other groups, each with a length of its own
    rng = random.Random(9)
    pages, pool, lens = case(40, 12, 16, 4, 3)
    parents = [rng.randrange(40) for _ in range(40)]
    run(pages, pool, parents, [rng.randint(0, lens[p]) for p in parents], [0, 7, 7, 25, 40])
    status()
    holders_of(pages)


def test_take_back_and_free():
    pages, pool, lens = case(6, 10, 16, 3, 5)
    run(pages, pool, list(range(6)), [max(1, n // 2) for n in lens])  # the last tokens go
    run(pages, pool, list(range(6)), [max(1, n // 2) for n in lens])  # nothing to do
    run(pages, pool, [-1] * 6, [0] * 6)
    status()
    holders_of(pages)
    assert pages.owned.tolist() == [0] * 6


def test_page_that_others_hold_too():
    # a program keeps a prompt's pages itself: they stay when the last request is gone
    pages = KVPages.create(8, 16, 2, 4, shared=True)
    step = pages.step(40, max_new=40)
    lens = dev([0, 0], torch.int32)
    pages.plan(lens, dev([40, 0], torch.int32), step)
    kept = pages.tables[0, :2].tolist()
    pages.shares[kept] += 1
    copies = pages.fork(dev([0, 0], torch.int32), dev([40, 40], torch.int32))
    assert pages.shares[kept].tolist() == [2, 2] and copies.rows.tolist() == [0, 8]
    pages.fork(dev([-1, -1], torch.int32), lens)
    status()
    assert pages.shares[kept].tolist() == [0, 0] and pages.owned.tolist() == [0, 0]
    head, tail = pages.ring_state.tolist()
    assert tail - head == 6
    # and a last, partly filled page that the program keeps is not written to
    pages.fork(dev([-1, -1], torch.int32), lens)
    pages.plan(lens, dev([8, 0], torch.int32), step)
    p = int(pages.tables[0, 0])
    pages.shares[p] += 1
    copies = pages.fork(dev([0, -1], torch.int32), dev([8, 0], torch.int32))
    status()
    assert copies.src.tolist() == [p, -1] and int(pages.tables[0, 0]) == int(copies.dst[0]) != p
    assert int(pages.shares[p]) == 0


def test_ring_runs_out():
    pages, pool, lens = case(4, 3, 16, 4, 8)
    pages.ring_state[1] = pages.ring_state[0] + 1  # one free page is left
    pool.tail = pool.head + 1
    n = 16 * min(pool.owned) - 3
    run(pages, pool, [0, 0, 0, 0], [n] * 4)
    assert sum(t[-(-n // 16) - 1] == -1 for t in pool.tables) == 2
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 3


@pytest.mark.parametrize("parents,lens", [([0, 1, 2, 5], [1, 1, 1, 1]), ([0, -2, 2, 3], [1, 1, 1, 1]),
                                          ([0, 1, 2, 3], [1, -1, 1, 1]), ([0, 1, 2, 3], [1, 1, 1 << 30, 1])])
def test_what_does_not_fit_is_cut_and_reported(parents, lens):
    pages, pool, _ = case(4, 3, 16, 2, 2)
    run(pages, pool, parents, lens, [0, 2, 4])
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 2


def test_absent_pages_and_strided_tables():
    pages, pool, lens = case(6, 9, 16, 3, 4)
    pool.tables[1][0] = pool.tables[4][2] = -1
    pool.tables[5][1] = 1 << 20
    for r, c in ((1, 0), (4, 2), (5, 1)):  # pages that no one holds now
        p = int(pages.tables[r, c])
        if p >= 0 and c < pool.owned[r]:
            pages.shares[p] -= 1
            pool.shares[p] -= 1
    wide = torch.full((6, 14), 12345, dtype=torch.int32, device="cuda")
    wide[:, 2:11] = dev(pool.tables, torch.int32)
    pages.tables = wide[:, 2:11]
    run(pages, pool, [1, 1, 2, 4, 5, 5], lens, [0, 3, 6])
    status()
    assert (wide[:, :2] == 12345).all() and (wide[:, 11:] == 12345).all()


def test_in_a_graph_and_on_another_stream():
    pages, pool, lens = case(8, 20, 16, 4, 6)
    parents, at, copies = dev([0] * 8, torch.int32), dev(lens, torch.int32), KVCopies.empty(8)
    prefix = KVPrefix.create(2, 4)
    first = [t.clone() for t in (pages.tables, pages.owned, pages.ring, pages.ring_state, pages.shares)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    pages.fork(parents, at, copies, prefix=prefix, stream=stream)
    stream.synchronize()
    for t, f in zip((pages.tables, pages.owned, pages.ring, pages.ring_state, pages.shares), first):
        t.copy_(f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pages.fork(parents, at, copies, prefix=prefix)
    rng = random.Random(2)
    for _ in range(4):
        new = [rng.randrange(a, a + 4) for a in (0, 4) for _ in range(4)]
        parents.copy_(dev(new, torch.int32))
        want = pool.fork(new, lens, [0, 4, 8])
        graph.replay()
        torch.cuda.synchronize()
        assert pages.tables.tolist() == pool.tables and pages.shares.tolist() == pool.shares
        assert (copies.src.tolist(), copies.dst.tolist(), copies.rows.tolist(), prefix.lens.tolist()) == want[1:]
        lens = want[0]
        at.copy_(dev(lens, torch.int32))
    status()


def test_plan_goes_on_from_forked_pages():
    # a prompt, four beams, and tokens of their own: no page that is written to is shared
    pages = KVPages.create(64, 16, 4, 16, shared=True)
    step = pages.step(50, max_new=50)
    lens = dev([0] * 4, torch.int32)
    pages.plan(lens, dev([45, 0, 0, 0], torch.int32), step)
    lens = dev([45] * 4, torch.int32)
    rng = random.Random(1)
    parents = [0, 0, 0, 0]
    copies = None
    for i in range(40):
        copies = pages.fork(dev(parents, torch.int32), lens, copies, lens_out=lens)
        pages.plan(lens, dev([1] * 4, torch.int32), step)
        status()
        holders_of(pages)
        slots = step.slots.tolist()[:4]
        assert len(set(slots)) == 4 and all(int(pages.shares[s // 16]) == 0 for s in slots)
        lens = lens + 1
        parents = [rng.randrange(4) for _ in range(4)]
    with pytest.raises(ValueError):
        pages.plan(lens, dev([0] * 4, torch.int32), step, trim=True)


def test_fork_refuses():
    pages = KVPages.create(8, 16, 2, 4)
    two = dev([0, 1], torch.int32)
    with pytest.raises(ValueError, match="shares"):
        pages.fork(two, two)
    pages = KVPages.create(8, 16, 2, 4, shared=True)
    for bad in (dict(parents=two.long()), dict(parents=two[:1]), dict(lens=two.cpu()), dict(lens_out=two[:1]),
                dict(copies=KVCopies.empty(3)), dict(prefix=KVPrefix(two, dev([0], torch.int32)))):
        with pytest.raises(ValueError):
            pages.fork(**{**dict(parents=two, lens=two), **bad})
    with pytest.raises(TypeError):
        pages.fork([0, 1], two)
    with pytest.raises(ValueError):
        KVPages(pages.tables, pages.owned, pages.ring[:4], pages.ring_state, 16, shares=pages.shares)
    with pytest.raises(ValueError):
        KVCopies(two, two[:1])
    with pytest.raises(ValueError):
        KVPrefix(two[:1], two)
    assert pages.ring_state.tolist() == [0, 8]


# ---------------------------------------------------------------- copy
@pytest.mark.parametrize("layout", ["hnd", "nhd", "gap"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (128, 3, 48), (256, 2, 64), (128, 8, 128)])
def test_copy(dim, heads, page, q8, layout):
    g = torch.Generator(device="cuda").manual_seed(dim + page)
    caches = []
    for _ in range(3):
        c = make_cache(23, heads, page, dim, q8, layout)
        for t in (c.k, c.v):
            t.copy_(torch.randint(-100, 100, t.shape, device="cuda", generator=g))
        if q8:
            c.scales.copy_(torch.rand(c.scales.shape, device="cuda", generator=g))
        caches.append(c)
    bits = [[t.clone() for t in (c.k, c.v, c.scales) if t is not None] for c in caches]
    src, dst = [3, -1, 5, 5, 9, 22, 0], [1, 2, -1, 4, 7, 21, 8]
    for rows in (None, [1, 5, 5, page, page - 1, 17 % page, 0], [page + 9, 2, 2, 15, 16, -3, 1]):
        copies = KVCopies(dev(src, torch.int32), dev(dst, torch.int32), None if rows is None else dev(rows, torch.int32))
        caches[0].copy(copies, others=caches[1:])
        status()
        for c, held in zip(caches, bits):
            for t, want in zip([x for x in (c.k, c.v, c.scales) if x is not None], held):
                for i, (a, b) in enumerate(zip(src, dst)):
                    n = page if rows is None else max(0, min(rows[i], page))
                    if a >= 0 and b >= 0:
                        want[b, :, :n] = want[a, :, :n]
                assert torch.equal(t, want)


def test_copy_of_bits_that_are_no_numbers():
    c = make_cache(4, 2, 16, 64, False)
    c.k.view(torch.int16).copy_(torch.randint(-32768, 32767, c.k.shape, device="cuda", dtype=torch.int16))
    c.v.fill_(float("nan"))
    c.copy(KVCopies(dev([1], torch.int32), dev([2], torch.int32)))
    status()
    assert torch.equal(c.k[1].view(torch.int16), c.k[2].view(torch.int16))


def test_copy_many_layers_and_pages():
    caches = [make_cache(70, 1, 16, 64, False) for _ in range(70)]  # more than one launch takes
    for i, c in enumerate(caches):
        c.k[:35], c.v[:35] = i + 1, -i - 1
        c.k[35:], c.v[35:] = 0, 0
    order = torch.randperm(35)
    caches[0].copy(KVCopies(order.int().cuda(), (35 + torch.arange(35)).int().cuda()), others=caches[1:])
    status()
    assert all((c.k[35:] == i + 1).all() and (c.v[35:] == -i - 1).all() for i, c in enumerate(caches))


def test_copy_reports_pages_outside():
    c = make_cache(4, 2, 16, 64, False)
    c.k.zero_(), c.v.zero_()
    c.k[1] = 1
    c.copy(KVCopies(dev([1, 1, 4], torch.int32), dev([4, 2, 3], torch.int32)))
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 1
    assert (c.k[2] == 1).all() and (c.k[3] == 0).all()


def test_copy_refuses():
    a, b = make_cache(4, 2, 16, 64, False), make_cache(5, 2, 16, 64, False)
    one = dev([0], torch.int32)
    with pytest.raises(w12.W12Error) as e:
        a.copy(KVCopies(one, dev([1], torch.int32)), others=[b])
    assert e.value.status == 2
    with pytest.raises(TypeError):
        a.copy(KVCopies(one, one), others=3)
    a.copy(KVCopies(one[:0], one[:0]))  # nothing to do
    status()
