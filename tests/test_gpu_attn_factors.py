"""GPU: factors of the scores at the ends of fp32."""
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


@pytest.mark.parametrize("kv,new", [([70], [1]), ([70], [2]), ([300], [200])])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_scale_of_nothing(kv, new, dtype):
    """A scale at the very end of fp32: every visible key weighs alike, and keys that are masked stay so."""
    cache, table, refs = build(kv, 1, 64, 16, "Q8_0", "Q8_0", 13)
    q = torch.randn(new[0], 2, 64, generator=torch.Generator().manual_seed(3)).to(TYPES[dtype])
    out = ft.attn_kv(cache, q.cuda(), table, ints(kv), ints([0, new[0]]), scale=1e-45)
    o, terms, bias, mass = kv_ref.attention(q.double().numpy(), *refs[0], new[0], kv[0], scale=1e-45)
    bound = kv_ref.attention_bound(o, terms, bias, mass, refs[0][1], dtype)
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= bound)
