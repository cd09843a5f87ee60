"""CPU tests of calls on tensors of a GPU that is not the current one: the library launches on the current
GPU, so they are refused before anything is enqueued."""
import pytest
import torch

from bit_affine_quantized_qmv_amd import api, kv


class OnGpu:
    """What the stream's lookup asks of a tensor."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


@pytest.fixture
def two_gpus(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(api, "_gpus", 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: type("S", (), {"cuda_stream": 1000 + device.index}))


def test_streams_of_the_current_gpu(two_gpus):
    assert kv.raw_stream(OnGpu(1)) == 1001 and api._stream(torch.device("cuda:1")) == 1001


def test_streams_of_another_gpu_are_refused(two_gpus):
    for _ in range(2):
        with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
            kv.raw_stream(OnGpu(0))
        with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
            api._stream(torch.device("cuda:0"))
