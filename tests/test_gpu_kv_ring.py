"""A ring of free pages without room for what a trimming plan gives back."""
import random

import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVPages, w12
from test_gpu_kv import dev, plan_case, plan_ref, run_plan, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def short_ring_ref(lens, new, owned, tables, ring, state, page, blocks):
    """plan with trim, one request at a time: a request gives back the last of its pages
    too many, as many as the ring still has room for."""
    n, size = len(lens), len(ring)
    tables, ring, (head, tail) = [list(r) for r in tables], list(ring), state
    src, avail = list(ring), tail - head
    room, taken, back, owned_out = size - avail, 0, 0, []
    for b in range(n):
        need, have = -(-(lens[b] + new[b]) // page), owned[b]
        for j in range(have, need):
            tables[b][j] = src[(head + taken) % size] if taken < avail else -1
            have += taken < avail
            taken += 1
        give = min(max(have - need, 0), room - back)
        for j in range(have - give, have):
            ring[(tail + back) % size] = tables[b][j]
            back += 1
        owned_out.append(have - give)
    return tables, owned_out, ring, [head + min(taken, avail), tail + back]


def short_ring_case(n, blocks, page, size, free, seed):
    rng = random.Random(seed)
    ids = list(range(n * blocks + free))
    rng.shuffle(ids)
    owned = [rng.randint(0, blocks) for _ in range(n)]
    lens = [rng.randint(0, min(blocks, have + 1)) * page if rng.random() < 0.7 else 0 for have in owned]
    tables, at = [], free
    for have in owned:
        tables.append(ids[at:at + have] + [-1] * (blocks - have))
        at += have
    head = rng.randrange(1 << 33)
    ring = [-7] * size
    for i in range(free):
        ring[(head + i) % size] = ids[i]
    return lens, [0] * n, owned, tables, ring, [head, head + free]


# one CTA; the cluster; several chunks of requests
@pytest.mark.parametrize("n,blocks,size,free,tokens", [(3, 9, 6, 5, 8), (40, 6, 50, 50, 8), (40, 6, 50, 17, 8),
                                                       (400, 8, 300, 120, 4096), (2300, 4, 2000, 1999, 5000),
                                                       (2300, 4, 900, 300, 8)])
@pytest.mark.parametrize("in_place", [True, False])
def test_pages_without_room_stay_with_their_requests(n, blocks, size, free, tokens, in_place):
    page = 16
    case = short_ring_case(n, blocks, page, size, free, seed=n + free)
    got = run_plan(case, page, tokens, True, in_place)
    want = short_ring_ref(*case, page, blocks)
    for g, w, what in zip(got, want, ("tables", "owned", "ring", "ring_state")):
        assert g == w, what
    assert got[3][1] - case[5][0] <= size  # never more than there is room for
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 3
    w12.w12_check_status()


def test_kept_pages_go_back_when_there_is_room_again():
    pages = KVPages(dev([[4, 5, 6, 7], [8, 9, -1, -1]], torch.int32), dev([4, 2], torch.int32),
                    dev([1, 2, 3, -1], torch.int32), dev([4, 7], torch.int64), 16)
    step, none, zero = pages.step(64), dev([0, 0], torch.int32), dev([0, 0], torch.int32)
    pages.plan(zero, none, step, trim=True)
    with pytest.raises(w12.W12Error):
        w12.w12_check_status()
    assert pages.owned.tolist() == [3, 2] and pages.ring_state.tolist() == [4, 8]
    assert pages.ring.tolist() == [1, 2, 3, 7]
    pages.plan(dev([64, 0], torch.int32), none, step)  # one page is taken, in request order
    assert pages.owned.tolist() == [4, 2] and pages.tables.tolist()[0] == [4, 5, 6, 1]
    pages.plan(dev([64, 16], torch.int32), none, step, trim=True)
    assert pages.owned.tolist() == [4, 1] and pages.ring_state.tolist() == [5, 9]
    assert sorted(pages.ring.tolist()) == [2, 3, 7, 9]
    status()


@pytest.mark.parametrize("state", [[5, 4], [3, 14]])
def test_state_that_is_no_ring_is_reported(state):
    """tail - head below 0 or above the ring's length."""
    pages = KVPages(dev([[0, 1]], torch.int32), dev([2], torch.int32), dev(list(range(10)), torch.int32),
                    dev(state, torch.int64), 16)
    step = pages.step(4)
    pages.plan(dev([16], torch.int32), dev([0], torch.int32), step)
    assert pages.owned.tolist() == [2] and pages.ring_state.tolist() == state
    with pytest.raises(w12.W12Error) as e:
        w12.w12_check_status()
    assert e.value.status == 3


def test_full_ring_is_no_fault():
    """Every page given back at once into a ring of as many entries."""
    case = plan_case(30, 200, 3, 16, 16, True, seed=8)
    lens, add, owned, tables, ring, (head, tail) = case
    lens, add = [0] * 30, [0] * 30
    case = (lens, add, owned, tables, ring, [head, tail])
    got, want = run_plan(case, 16, 100, True), plan_ref(*case, 16, 16, 100, True)
    assert got == want and got[1] == [0] * 30
    assert got[3][1] - got[3][0] == (tail - head) + sum(owned)
    status()
