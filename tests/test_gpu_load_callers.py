"""GPU: forms of ft.kv_load's arguments that its callers use."""
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

T, H, D = 5, 2, 64


@pytest.fixture
def stored():
    """A cache whose first T slots hold 127, and their slots."""
    need_gpu()
    cache, slots = ft.KvCache.empty(2, 16, H, D), torch.arange(T, device="cuda")
    x = torch.full((T, H, D), 127.0, device="cuda")
    ft.kv_store(cache, x, x, slots)
    return cache, slots


@pytest.mark.parametrize("side", ["k", "v"])
def test_a_given_side_decides_the_type(stored, side):
    """dtype is read only where neither side is given: None, or another type, beside a given one."""
    for dtype in (None, torch.float32, torch.float64):
        mine = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
        k, v = ft.kv_load(*stored, dtype=dtype, **{side: mine})
        assert (k if side == "k" else v) is mine and k.dtype is v.dtype is torch.bfloat16
        assert torch.equal(k, torch.full_like(k, 127.0)) and torch.equal(v, k)
    with pytest.raises(ValueError, match="dtype must be"):
        ft.kv_load(*stored, dtype=None)


class Handle:
    """A stream as its device and handle, and nothing else."""

    def __init__(self, stream):
        self.device, self.cuda_stream = stream.device, stream.cuda_stream


def test_a_stream_is_its_device_and_handle(stored):
    cache, slots = stored
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    k, v = ft.kv_load(cache, slots, stream=Handle(stream))
    stream.synchronize()
    assert torch.equal(k, torch.full_like(k, 127.0)) and torch.equal(v, k)
    elsewhere = Handle(stream)
    elsewhere.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="the stream is on"):
        ft.kv_load(cache, slots, stream=elsewhere)
