"""GPU: forms of ft.kv_load's arguments that its callers use."""
import sys

import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu, own_stream

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
    stream = own_stream()
    k, v = ft.kv_load(cache, slots, stream=Handle(stream))
    stream.synchronize()
    assert torch.equal(k, torch.full_like(k, 127.0)) and torch.equal(v, k)
    elsewhere = Handle(stream)
    elsewhere.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="the stream is on"):
        ft.kv_load(cache, slots, stream=elsewhere)


def test_the_library_alone_is_enough(stored, monkeypatch):
    """Without the compiled marshalling (a package with libft.so only) rows are read back all the same, and refused the same way."""
    want = ft.kv_load(*stored, dtype=torch.bfloat16)
    monkeypatch.setattr(ft, "_ext", None)
    monkeypatch.setitem(sys.modules, "block_quantized_matvec_amd._ft_bind", None)
    monkeypatch.delattr("block_quantized_matvec_amd._ft_bind", raising=False)
    with pytest.raises(RuntimeError, match="does not load"):
        ft.norm(torch.ones(2, 32, device="cuda"))
    cache, slots = stored
    for kw in (dict(dtype=torch.bfloat16), dict(k=want[0].clone()), dict(dtype=None, v=want[1].clone()), dict(dtype=torch.bfloat16, stream=torch.cuda.current_stream())):
        got = ft.kv_load(cache, slots, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(g is kw[n] for n, g in zip("kv", got) if n in kw)
    for bad in (dict(dtype=torch.float64), dict(dtype=None), dict(k=want[0][:2]), dict(v=want[1].cpu())):
        with pytest.raises(ValueError):
            ft.kv_load(cache, slots, **bad)
    with pytest.raises((ValueError, ft.FtError)):
        ft.kv_load(cache, slots.int())
