"""What the Python calls ask of the rank tensors before they take any
address: host only."""

import pytest
import torch

pytest.importorskip("gradient_all_reduce_allreduce_amd")
from gradient_all_reduce_allreduce_amd import api  # noqa: E402


class Elsewhere(torch.Tensor):
    """A tensor on numbered device 0 of another kind than the GPU."""
    is_cuda = False

    def get_device(self):
        return 0


class OnGpu(Elsewhere):
    is_cuda = True


def make(kind, n=4, dtype=torch.float32):
    return torch.Tensor._make_subclass(kind, torch.zeros(n, dtype=dtype))


def test_a_device_number_does_not_make_a_gpu_tensor():
    for ts in ([make(Elsewhere)] * 2, [make(OnGpu), make(Elsewhere)], [make(Elsewhere), make(OnGpu)],
               [torch.zeros(4)], [make(OnGpu), torch.zeros(4)]):
        with pytest.raises(ValueError, match="must live on the GPU"):
            api._rank_tensors(ts, "ranks")


def test_equal_gpu_tensors_pass():
    ts = [make(OnGpu), make(OnGpu)]
    assert api._rank_tensors(iter(ts), "ranks") == ts
    for other in (make(OnGpu, 5), make(OnGpu, 4, torch.bfloat16)):
        with pytest.raises(ValueError, match="same device, dtype and size"):
            api._rank_tensors([ts[0], other], "ranks")
    with pytest.raises(ValueError, match="contiguous"):
        api._rank_tensors([torch.Tensor._make_subclass(OnGpu, torch.zeros(4, 4).t())], "ranks")
