"""Two host threads whose attention calls share a stream, and so its workspace."""
import threading

import pytest
import torch

from test_gpu_kv import attend_case, attend_ref, check_attend, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gpu_util import ensure_built
    ensure_built()


# one shape for both threads, two shapes of the same kernels, and with the tcgen05 kernel
@pytest.mark.parametrize("groups", [(6, 6), (6, 3), (6, 40)])
def test_two_threads_on_one_stream(groups):
    calls, dim = 3000, 128
    cases = []
    for seed, group in enumerate(groups):
        lens = [1500 + 200 * seed]
        cache, tables, cu, q, step = attend_case(lens, [1], group, 1, dim, 16, False, seed=seed)
        out, lse = run_attend(cache, q, step)  # by itself, and the workspace is large enough from here on
        check_attend(out, lse, attend_ref(q, cache, tables, lens, cu, None, 0, dim ** -0.5, group))
        outs = torch.zeros(calls, 1, group * dim, device="cuda", dtype=torch.bfloat16)
        cases.append((cache, q.view(1, -1), step, out, list(outs.unbind()), outs))
    torch.cuda.synchronize()
    gate, failed = threading.Barrier(len(cases)), []

    def work(cache, q, step, want, outs, _):
        try:
            gate.wait(30)
            for out in outs:
                cache.attend(q, step, out=out)
        except BaseException as e:  # noqa: BLE001 (the test's thread has to see it)
            failed.append(e)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed and not any(t.is_alive() for t in threads)
    torch.cuda.synchronize()
    for _, _, _, want, _, outs in cases:
        wrong = (outs != want).flatten(1).any(1)
        assert not wrong.any(), f"{int(wrong.sum())} of {calls} calls gave other bits"
