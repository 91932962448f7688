"""Calls that are the first CUDA work of their host thread."""
import threading

import pytest
import torch

from lossless_bit_weight_encode_gb300 import W12Weight, w12
from lossless_bit_weight_encode_gb300 import workloads as wl
from gpu_util import to_dev_bf16
from test_gpu_kv import attend_case, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


def in_thread(f):
    failed = []

    def run():
        try:
            f()
        except BaseException as e:  # noqa: BLE001 (the test's thread has to see it)
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join(60)
    assert not t.is_alive() and not failed, failed
    torch.cuda.synchronize()


@pytest.mark.parametrize("heads", [6, 40])  # the warp-level and the tcgen05 kernel
def test_attend(heads):
    cache, _, _, q, step = attend_case([700], [1], heads, 1, 128, 16, False, seed=heads)
    want, lse = run_attend(cache, q, step)
    out, lse2 = torch.zeros_like(want), torch.zeros_like(lse)
    q = q.view(1, -1)
    in_thread(lambda: cache.attend(q, step, out=out, lse=lse2))
    assert torch.equal(out, want) and torch.equal(lse2, lse)


@pytest.mark.parametrize("tokens", [1, 16])
def test_product(tokens):
    w = W12Weight(wl.gaussian_weights(700, 3000, seed=3))
    x = to_dev_bf16(wl.activations(tokens, 3000, seed=4))
    want = w.gemm(x)
    y, ws = torch.zeros_like(want), w.workspace(tokens)
    in_thread(lambda: w12.w12_gemm(x, w.blob, w.info, y, tokens, ws))
    w12.w12_check_status()
    assert torch.equal(y, want)
