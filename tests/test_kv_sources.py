"""What the paged-cache kernels' sources must not have.  (Text checks: the mistakes they
stand for show on a GPU only now and then.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bit_weight_encode_gb300",
                    "csrc")
KERNELS = sorted(f for f in os.listdir(CSRC) if f.startswith("kv_") and f.endswith(".cuh"))


@pytest.mark.parametrize("name", KERNELS)
def test_no_non_coherent_loads(name):
    """These kernels may be resident while the one before them still writes q, the page
    tables and lengths: a load through the non-coherent path is defined only for memory
    that nothing writes during the kernel's whole life."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    hits = [m.group(0) for m in re.finditer(r"__ldg\b|\.global\.nc\b|const\s+\w+\s*\*\s*__restrict__", text)]
    assert not hits, f"{name}: {hits}"


def test_joining_kernel_fences_what_it_reads_before_it_waits():
    """Lengths and offsets alone, and those behind a fence: nothing else orders its loads
    with the writes of kernels that ended before it began."""
    with open(os.path.join(CSRC, "kv_attend.cuh")) as f:
        text = f.read()
    start = text.index("w12_kv_join_kernel(const KvAttendParams p, int grid)")
    ahead = text[start:text.index("pdl_wait();", start)]
    loads = [m.start() for m in re.finditer(r"p\.(cu_new|lens)\[|kv_request<|kv_sum_units<", ahead)]
    assert loads and "__threadfence();" in ahead[:min(loads)]
    assert not re.search(r"p\.(tables|tree|q|part|part_ml)\s*\[", ahead)
