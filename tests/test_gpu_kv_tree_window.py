"""Sliding windows over drafted trees: a token's place is its depth, not its number."""
import math
import random

import numpy as np
import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVStep
from test_gpu_kv import attend_case, attend_ref, check_attend, dev, held_rows, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def draw_trees(new, seed):
    """(masks, depths): each token's ancestors and itself, and how deep it is."""
    rng = random.Random(seed)
    masks, depths = [], []
    for n in new:
        m, d = [], []
        for i in range(n):
            parent = rng.randrange(max(0, i - 6), i) if i and i < 32 else min(i, 31) - 1 if i else -1
            m.append((m[parent] if parent >= 0 else 0) | (1 << i if i < 32 else 0))
            d.append(d[parent] + 1 if parent >= 0 else 0)
        masks += m
        depths += d
    return masks, depths


def tree_window_ref(q, cache, tables, lens, cu, masks, places, window, scale, group):
    """As attend_ref, with the window between the tokens' places: a cached key's is its
    index, a new token's is given."""
    t, h, dim = q.shape
    out = torch.zeros(t, h, dim, dtype=torch.float64)
    mass, lse, big = out.clone(), torch.full((t, h), -math.inf, dtype=torch.float64), torch.zeros(t, h, dtype=torch.float64)
    q = q.double().cpu()
    for b, past in enumerate(lens):
        m = cu[b + 1] - cu[b]
        k, v, ok = held_rows(cache, tables[b], past + m)
        place = torch.tensor(list(range(past)) + places[cu[b]:cu[b + 1]], dtype=torch.int64)
        for i in range(m):
            bits = masks[cu[b] + i]
            drawn = torch.tensor([j < past or (j - past < 32 and bits >> (j - past) & 1 == 1) for j in range(past + m)],
                                 dtype=torch.bool)
            see = ok & drawn & (place > places[cu[b] + i] - window)
            if not see.any():
                continue
            kk, vv = (x[see].repeat_interleave(group, 1) for x in (k, v))
            row = q[cu[b] + i]
            s = torch.einsum("hd,khd->hk", row, kk) * scale
            w = torch.softmax(s, -1)
            out[cu[b] + i] = torch.einsum("hk,khd->hd", w, vv)
            mass[cu[b] + i] = torch.einsum("hk,khd->hd", w, vv.abs())
            lse[cu[b] + i] = torch.logsumexp(s, -1)
            big[cu[b] + i] = (torch.einsum("hd,khd->hk", row.abs(), kk.abs()) * scale).amax(-1)
    return out, lse, mass, big


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 2, 2), (128, 6, 2), (128, 1, 1), (256, 6, 1), (64, 20, 2)])
@pytest.mark.parametrize("window", [1, 2, 5, 17, 40, 100, 1 << 20])
def test_window_goes_by_depth(q8, dim, heads, kv_heads, window):
    lens, new = [0, 100, 48, 7, 63], [6, 16, 32, 1, 36]
    if heads == kv_heads:  # up to 16 rows: the warp-level kernel
        new = [6, 8, 7, 1, 8]
    cache, tables, cu, q, step = attend_case(lens, new, heads, kv_heads, dim, 16, q8, seed=dim + heads)
    masks, depths = draw_trees(new, seed=window)
    places = [past + d for b, past in enumerate(lens) for d in depths[cu[b]:cu[b + 1]]]
    step.tree = torch.from_numpy(np.array(masks, np.uint32).view(np.int32)).cuda()
    step.positions = dev(places, torch.int32)
    out, lse = run_attend(cache, q, step, window=window)
    check_attend(out, lse, tree_window_ref(q, cache, tables, lens, cu, masks, places, window, dim ** -0.5,
                                           heads // kv_heads))


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (24, 2)])
def test_path_of_a_tree_sees_what_decoding_it_sees(heads, kv_heads):
    """Tokens 0, 2, 5 of a branching tree, and the same three as a chain."""
    past, dim, window = 200, 128, 20
    cache, tables, cu, q, step = attend_case([past], [6], heads, kv_heads, dim, 16, False, seed=9)
    step.tree = dev([1, 3, 5, 11, 19, 37], torch.int32)  # 0; 0-1; 0-2; 0-1-3; 0-1-4; 0-2-5
    step.positions = dev([200, 201, 201, 202, 202, 202], torch.int32)
    out, lse = run_attend(cache, q, step, window=window)
    path, scale, group = [0, 2, 5], dim ** -0.5, heads // kv_heads
    ref = tree_window_ref(q, cache, tables, [past], cu, [1, 3, 5, 11, 19, 37], step.positions.tolist(), window, scale,
                          group)
    check_attend(out, lse, ref)
    slots = dev([int(tables[0, (past + i) // 16]) * 16 + (past + i) % 16 for i in range(6)], torch.int64)
    k, v = cache.read(slots)
    cache.store(None, k[path].contiguous(), v[path].contiguous(), KVStep(slots=slots[:3].contiguous()))
    chain = KVStep(step.tables, step.lens, dev([0, 3], torch.int32), max_new=3)
    out, lse = run_attend(cache, q[path].contiguous(), chain, window=window)
    want = attend_ref(q[path], cache, tables, [past], [0, 3], None, window, scale, group)
    check_attend(out, lse, want)
    assert (ref[0][path] - want[0]).abs().max() < 1e-12  # the same keys and weights


@pytest.mark.parametrize("heads", [2, 20])
def test_places_are_held_between_past_and_number(heads):
    """Below the cached length or above lens + number a place counts as the nearest."""
    lens, new, dim = [50, 70], [5, 8], 64
    cache, tables, cu, q, step = attend_case(lens, new, heads, 1, dim, 16, False, seed=4)
    masks, _ = draw_trees(new, seed=1)
    wild = [0, 10, 1 << 30, -5, 53, -(1 << 31), 71, 500, 2 ** 31 - 1, 0, 75, 74, 3]
    places = [min(max(wild[t], lens[b]), lens[b] + t - cu[b]) for b in (0, 1) for t in range(cu[b], cu[b + 1])]
    step.tree = torch.from_numpy(np.array(masks, np.uint32).view(np.int32)).cuda()
    step.positions = dev(wild, torch.int32)
    for window in (3, 12):
        out, lse = run_attend(cache, q, step, window=window)
        check_attend(out, lse, tree_window_ref(q, cache, tables, lens, cu, masks, places, window, dim ** -0.5, heads))


def test_places_matter_to_windowed_trees_alone():
    lens, new, dim = [50, 70], [5, 8], 64
    cache, tables, cu, q, step = attend_case(lens, new, 4, 2, dim, 16, False, seed=5)
    step.positions = dev([0] * 3, torch.int32)  # not even one per token
    out, lse = run_attend(cache, q, step, window=9)  # no tree: tokens are numbered
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, 9, dim ** -0.5, 2))
    masks, _ = draw_trees(new, seed=3)
    tree = np.array(masks, np.uint32).view(np.int32)
    step.tree = torch.from_numpy(tree).cuda()
    out, lse = run_attend(cache, q, step)  # no window
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, tree, 0, dim ** -0.5, 2))
    with pytest.raises(ValueError):
        cache.attend(q.view(13, -1), step, window=9)
    step.positions = None  # numbers again
    out, lse = run_attend(cache, q, step, window=9)
    check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, tree, 9, dim ** -0.5, 2))
