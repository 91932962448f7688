"""Paged-cache calls at the ends of their ranges."""
import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVPages, w12
from test_gpu_kv import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


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
