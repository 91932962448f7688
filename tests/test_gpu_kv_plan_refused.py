"""A plan that is refused leaves its step as it was."""
import pytest
import torch

from lossless_bit_weight_encode_gb300 import KVPages
from test_gpu_kv import dev, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("stream", [None, "side"])
def test_step_keeps_its_lengths_and_tables(stream):
    pages, others = (KVPages.create(8, 16, requests=2, max_blocks=4) for _ in range(2))
    step, lens, new = pages.step(40), dev([0, 0], torch.int32), dev([20, 9], torch.int32)
    s = torch.cuda.Stream() if stream else None
    assert pages.plan(lens, new, step, stream=s) is step
    assert step.lens is lens and step.tables is pages.tables
    longer = dev([20, 9], torch.int32)
    for bad in (new[:1], new.float(), dev([1, 1, 1], torch.int32)):
        with pytest.raises(ValueError):
            others.plan(longer, bad, step, stream=s)
        assert step.lens is lens and step.tables is pages.tables
    with pytest.raises(ValueError):
        pages.plan(longer[:1], new, step, stream=s)
    assert step.lens is lens
    pages.plan(longer, new, step, stream=s)
    assert step.lens is longer
    status()
    assert pages.owned.tolist() == [3, 2]
