"""GPU: attention whose keys are split over workgroups: parts that hold no key, more parts than a wave joins at once,
captured calls whose lengths grow over the borders of the parts."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import need_gpu
from tests.test_gpu_attn_kv import TYPES, build, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def right(out, q, kv, new, refs, dtype, **kw):
    out, q = out.double().cpu().numpy(), q.double().cpu().numpy()
    start = np.concatenate([[0], np.cumsum(new)])
    for i, (n, c) in enumerate(zip(kv, new)):
        a = slice(start[i], start[i + 1])
        o, terms, bias, mass = kv_ref.attention(q[a], refs[i][0][:n], refs[i][1][:n], c, n, **kw)
        bound = kv_ref.attention_bound(o, terms, bias, mass, refs[i][1][:n], dtype)
        assert np.all(np.isfinite(out[a])) and np.all(np.abs(out[a] - o) <= bound), (i, n)


def wide(table, cols):
    t = torch.zeros(table.shape[0], cols, dtype=torch.int32, device="cuda")
    t[:, :table.shape[1]] = table
    return t


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("kv,new,max_kv", [([200], [150], 20000), ([90, 1, 200], [90, 1, 60], 9000), ([70], [3], 30000), ([0, 64], [1, 1], 30000)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_parts_without_keys(kv, new, max_kv, dim, dtype):
    """A host bound far above the lengths: most workgroups have nothing to do and say so."""
    cache, table, refs = build(kv, 2, dim, 16, "Q8_0", "Q8_0", 21)
    q = torch.randn(sum(new), 8, dim, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    args = (cache, q.cuda(), wide(table, -(-max_kv // 16)), ints(kv), ints(np.concatenate([[0], np.cumsum(new)])))
    assert ft.attn_kv_scratch_bytes(cache, sum(new), 8, len(new), max_kv) > 0
    right(ft.attn_kv(*args, max_kv=max_kv), q, kv, new, refs, dtype)
