"""GPU: a row whose scores are not numbers says so (NaN throughout), whether or not its keys are split, and no other
row does."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu
from tests.test_gpu_attn_kv import TYPES, build, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# the kernel for few rows (whole, eight waves, split) and the one for many (whole, split), a shared prefix in both
@pytest.mark.parametrize("kv,new,max_kv,shared", [([50], [3], 50, 0), ([400], [3], 400, 0), ([3000, 40], [1, 2], 3000, 0), ([40], [3], 9000, 0),
                                                  ([200], [150], 200, 0), ([2900], [150], 3000, 0), ([300, 2500], [90, 1], 2500, 0),
                                                  ([200, 180], [1, 2], 200, 128), ([400, 390], [140, 130], 400, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_not_a_number(kv, new, max_kv, shared, value, dtype):
    heads = 6
    cache, table, _ = build(kv, 2, 64, 16, "Q8_0", "Q8_0", 11, shared)
    wide = torch.zeros(len(kv), -(-max_kv // 16), dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = torch.randn(sum(new), heads, 64, generator=torch.Generator().manual_seed(2)).to(TYPES[dtype]).cuda()
    args = (wide, ints(kv), ints(np.concatenate([[0], np.cumsum(new)])))
    clean = ft.attn_kv(cache, q, *args, max_kv=max_kv, n_shared=shared)
    assert torch.isfinite(clean).all()
    bad = torch.zeros(sum(new), heads, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[-1, heads - 1] = bad[sum(new) // 2, 3] = True
    broken = q.clone()
    broken[0, 1, 5] = broken[-1, heads - 1, 63] = broken[sum(new) // 2, 3, 32] = value
    out = ft.attn_kv(cache, broken, *args, max_kv=max_kv, n_shared=shared)
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_not_a_number_without_keys(dtype):
    """A row that sees nothing is zero, whatever it holds."""
    cache, table, _ = build([5, 70], 2, 64, 16, "Q8_0", "Q8_0", 12)
    q = torch.full((3, 4, 64), float("nan"), device="cuda", dtype=TYPES[dtype])
    out = ft.attn_kv(cache, q, table, ints([0, 70]), ints([0, 2, 3]))
    assert not out[:2].any() and torch.isnan(out[2]).all()
