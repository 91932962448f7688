"""Attention behind shared prefixes for many requests of 9 to 16 rows each, whose row tile is
another one than that of their few groups, against plain attention in 64 bits."""
import random

import pytest
import torch
from test_gpu_shared import compare, shared_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("most", [0, 1, 2, None])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("heads,new", [(96, 1), (48, 2)])
@pytest.mark.parametrize("requests", [120, 300])
def test_groups_of_more_than_max_says(requests, heads, new, q8, most):
    rng = random.Random(requests + heads)
    # a tile and less, and several tiles, which more than one block of the grid shares
    members = [(rng.choice([0, 1, 20, 63, 64, 65, 130, 700]), new) for _ in range(requests)]
    case = shared_case([(5, members[:-30]), (0, members[-30:-10]), (2, members[-10:])], heads, 8, 128, 16, q8, 31)
    if most is not None:  # None: as it is
        case[-1].prefix.max_requests = most
    compare(case)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_few_new_tokens_among_many_requests(dim):
    members = [(500, 1)] + [(30, 0)] * 119
    compare(shared_case([(5, members)], 96, 8, dim, 16, False, 32))
    compare(shared_case([(5, members[::-1])], 96, 8, dim, 16, False, 33))
    torch.cuda.synchronize()
