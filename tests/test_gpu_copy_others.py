"""A page copy's other caches, given in any way that a loop takes."""
import pytest
import torch
from test_gpu_kv import dev, make_cache, status

from lossless_bit_weight_encode_gb300 import KVCopies

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


@pytest.mark.parametrize("way", [list, tuple, iter, lambda c: (x for x in c), lambda c: {id(x): x for x in c}.values()])
@pytest.mark.parametrize("on_a_stream", [False, True])
def test_all_caches_are_copied(way, on_a_stream):
    caches = [make_cache(4, 2, 16, 64, False) for _ in range(3)]
    for c in caches:
        c.k.fill_(0), c.v.fill_(0)
        c.k[1], c.v[1] = 5, 6
    stream = torch.cuda.Stream() if on_a_stream else None
    if stream:
        stream.wait_stream(torch.cuda.current_stream())
    caches[0].copy(KVCopies(dev([1], torch.int32), dev([3], torch.int32)), others=way(caches[1:]), stream=stream)
    if stream:
        torch.cuda.current_stream().wait_stream(stream)
    status()
    assert all((c.k[3] == 5).all() and (c.v[3] == 6).all() for c in caches)
