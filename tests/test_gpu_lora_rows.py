"""GPU: low-rank adapters, the rows that they leave alone."""
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu
from tests.test_gpu_lora import case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [5, 70, 1500])
def test_rows_pass_through_to_the_bit(t):
    """Rows of no adapter, or of an adapter of rank 0, are y's own bits: a zero keeps its sign."""
    need_gpu()
    for n in (40, 4100):
        x, a, b, y, ids, sc = case(t, 64, n, 3, 16)
        y[:, ::3] = -0.0
        ids[:] = torch.arange(t, dtype=torch.int32) % 4 - 1
        ranks = torch.tensor([0, 16, 16], dtype=torch.int32, device="cuda")
        out = ft.lora(x, a, b, ids, y=y, scales=sc, ranks=ranks)
        kept = ids < 1
        same = torch.equal(out[kept].view(torch.int32), y[kept].view(torch.int32))
        assert same
        check(out, x, a, b, ids, y, sc, ranks)
