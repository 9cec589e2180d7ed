"""GPU: a scratch size that cannot be had is refused, and the calls after it are none the worse."""
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_too_much_scratch():
    need_gpu()
    x = torch.randn(5, 16, device="cuda")
    ids, w = ft.moe_route(x, 4)
    s = torch.cuda.Stream()
    with pytest.raises(ft.FtError):
        ft.scratch_reserve(1 << 50, stream=s)
    again = ft.moe_route(x, 4)
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)
    ft.scratch_reserve(1 << 20, stream=s)
    torch.cuda.synchronize()
