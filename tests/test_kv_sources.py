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
