"""Attention where queries, keys or values are not finite: a row that sees one is not
finite, however its keys are split over CTAs and joined, and no other row is touched."""
import math

import numpy as np
import pytest
import torch

from lossless_bit_weight_encode_gb300 import w12
from test_gpu_kv import attend_case, attend_ref, check_attend, run_attend

pytestmark = pytest.mark.gpu

# Requests, key heads, query heads per key head: few blocks of rows for the device's CTAs
# (their parts are joined by a second kernel, a warp or eight per row) or many (joined by
# the CTA that arrives last, where a range ends inside a block); 40 rows: tcgen05.
SPLITS = [pytest.param([4000], 1, 5, id="eight-warps"),
          pytest.param([777], 1, 5, id="one-long"),
          pytest.param([900 + 61 * b for b in range(24)], 2, 3, id="one-warp"),
          pytest.param([500 + 7 * b for b in range(150)], 4, 2, id="last-cta"),
          pytest.param([4000], 1, 40, id="tc-one"),
          pytest.param([300 + 61 * b for b in range(12)], 2, 40, id="tc-many")]


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def check_but(hit, out, lse, ref):
    """The rows outside `hit` against the reference; those in it are NaN throughout."""
    out, lse, hit = out.view(ref[0].shape).cpu(), lse.cpu(), hit.cpu()
    assert torch.isnan(out[hit]).all(), f"{int((~torch.isnan(out[hit])).sum())} elements of NaN rows are not NaN"
    assert torch.isnan(lse[hit]).all()
    keep = ~hit
    check_attend(out[keep], lse[keep], tuple(x[keep] for x in ref))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,kv_heads,group", SPLITS)
def test_query_that_is_not_a_number(lens, kv_heads, group, q8, dim):
    cache, tables, cu, q, step = attend_case(lens, [1] * len(lens), kv_heads * group, kv_heads, dim, 16, q8, seed=dim)
    ref = attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, group)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit.view(-1)[::4] = True
    q = q.clone()
    q[..., 3][hit] = math.nan
    out, lse = run_attend(cache, q, step)
    check_but(hit, out, lse, ref)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,kv_heads,group", SPLITS)
def test_run_of_keys_that_are_not_numbers(lens, kv_heads, group, q8, dim):
    # whole parts of a row have nothing else, and the first one none: all keys from the
    # 128th on, of every third request's last key head
    cache, tables, cu, q, step = attend_case(lens, [1] * len(lens), kv_heads * group, kv_heads, dim, 16, q8, seed=dim)
    ref = attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, group)
    hit = torch.zeros(len(lens), kv_heads, group, dtype=torch.bool)
    hit[::3, -1] = True
    for b in range(0, len(lens), 3):
        pages = torch.from_numpy(tables[b, 8:-(-(lens[b] + 1) // 16)]).cuda()
        if q8:
            cache.scales[pages, kv_heads - 1, :, 0] = math.nan
        else:
            cache.k[pages, kv_heads - 1, :, 5] = math.nan
    out, lse = run_attend(cache, q, step)
    check_but(hit.view(len(lens), -1), out, lse, ref)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("group", [3, 12])  # the warp-level and the tcgen05 kernel
def test_requests_behind_one_that_is_not_finite(dim, bad, q8, group):
    """A drafted token's key and value of one head: its own rows of that head are not
    finite, the rows of the requests around it are as if nothing was there."""
    lens, new = [21, 37, 90, 5], [3, 5, 2, 4]
    cache, tables, cu, q, step = attend_case(lens, new, 2 * group, 2, dim, 16, q8, seed=2)
    tree = np.array([1, 2, 4] + [1, 2, 5, 10, 0b10001] + [1, 3] + [1, 2, 5, 9], np.int32)
    step.tree = torch.from_numpy(tree).cuda()  # token 1 of request 1 is seen by its tokens 1 and 3 alone
    ref = attend_ref(q, cache, tables, lens, cu, tree, 0, dim ** -0.5, group)
    page, off = int(tables[1, 38 // 16]), 38 % 16
    if q8:
        cache.scales[page, 1, off] = bad
    else:
        cache.v[page, 1, off, 3:9] = bad
        cache.k[page, 1, off, 2] = bad
    out, lse = run_attend(cache, q, step)
    out = out.view(ref[0].shape)
    seen = torch.zeros(out.shape[:2], dtype=torch.bool)
    seen[[4, 6], group:] = True
    assert not torch.isfinite(out[seen.cuda()][:, 3:9]).any()
    check_attend(out[~seen.cuda()], lse[~seen.cuda()], tuple(x[~seen] for x in ref))
    w12.w12_check_status()
