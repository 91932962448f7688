"""The paged cache's holders on the host, with stand-ins for device tensors."""
import pytest

torch = pytest.importorskip("torch")

from lossless_bit_weight_encode_gb300.kv import KVStep  # noqa: E402


class Fake:
    """What KVStep looks at in a tensor."""

    def __init__(self, device, dtype=torch.int32):
        self.dtype, self.device, self.is_cuda = dtype, device, True

    def get_device(self):
        return self.device

    def dim(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_refused_array_leaves_the_step_as_it_was():
    step = KVStep()
    with pytest.raises(ValueError):
        step.lens = Fake(1, torch.int64)
    step.lens = Fake(0)  # device 1 is not the step's for the array that it refused
    assert step.lens.device == 0
    with pytest.raises(ValueError):
        step.cu_new = Fake(1)
    step.cu_new = Fake(0)
