"""What the binding passes on and refuses, without a GPU: tensors that say they are on one, and a
library that records its calls."""
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(xp, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib.calls


def test_append_passes_the_columns_of_its_table(calls):
    wide = gpu(3, 10, dtype=torch.int32)
    k = gpu(3, 2, 4, 8)
    xp.xp_cache_append(1, 0, k, k, wide[:, 4:8], gpu(3, dtype=torch.int32), stream=0)
    (_, args), = calls
    assert args[11:13] == (10, 4)          # rows 10 apart, 4 columns
