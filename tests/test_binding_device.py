"""The verification entry points launch on the current device: tensors of another one are refused on the host."""
import pytest

from speculative_sampling_verification_spec_gb300 import binding


class Tensor:
    """As much of a CUDA tensor as the first check reads."""

    def __init__(self, device):
        self.is_cuda, self.device_index = device is not None, device

    def get_device(self):
        return self.device_index


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    binding._check_cuda(Tensor(1), None, Tensor(1))
    for ts in ((Tensor(0),), (Tensor(1), Tensor(2)), (Tensor(1), None, Tensor(None))):
        with pytest.raises(ValueError):
            binding._check_cuda(*ts)
