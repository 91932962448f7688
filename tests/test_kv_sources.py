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


def test_joining_kernel_reads_past_l1_before_it_waits():
    """Before its wait it may read lengths and offsets alone, and those from L2."""
    with open(os.path.join(CSRC, "kv_attend.cuh")) as f:
        text = f.read()
    start = text.index("w12_kv_join_kernel(const KvAttendParams p, int grid)")
    ahead = text[start:text.index("pdl_wait();", start)]
    assert "pdl_wait" not in ahead and len(ahead) > 500
    assert not re.search(r"p\.(cu_new|lens|tables|tree|q|part|part_ml)\s*\[", ahead)
    assert all("true>" in call for call in re.findall(r"kv_(?:request|sum_units|length)<[^>]*>", ahead))
