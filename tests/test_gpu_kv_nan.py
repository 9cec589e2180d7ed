"""GPU: a NaN among the rows that are written into the cache has no magnitude: it decides no scale, and the other
elements of its block keep the codes they would have with a zero in its place."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ty", ["Q8_0", "Q4_0"])
@pytest.mark.parametrize("dim", [64, 96])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_nan_has_no_magnitude(ty, dim, dtype):
    need_gpu()
    page, t = 16, 40
    cache = ft.KvCache.empty(3, page, 1, dim, ty, ty)
    g = torch.Generator().manual_seed(dim)
    x = torch.randn(t, 1, dim, generator=g).to(dtype)
    nan = torch.zeros(t, 1, dim, dtype=torch.bool)
    for i in range(t - 1):
        nan[i, 0, i % 32] = True                    # at every place of a block
        if i % 3 == 0:
            nan[i, 0, (i * 7 + 5) % dim] = True
    nan[t - 1] = True                               # nothing but NaN
    slots = torch.arange(t)
    broken = x.masked_fill(nan, float("nan")).cuda()
    ft.kv_store(cache, broken, broken, slots.cuda())
    q, d = kv_ref.quantize(x.masked_fill(nan, 0.0).float().numpy(), ty)
    for side, pool in (("k", host(cache.k_pages)), ("v", host(cache.v_pages))):
        for i in range(t):
            gq, gd = kv_ref.read_slot(pool, ty, side, page, 1, dim, i)
            assert np.array_equal(gd.view(np.uint16), d[i].view(np.uint16)), (side, i)
            keep = ~nan[i].numpy()
            assert np.array_equal(gq[keep], q[i][keep]), (side, i)
