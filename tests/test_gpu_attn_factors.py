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


@pytest.mark.parametrize("kv,new,dim", [([300], [2], 64), ([2000, 90], [1, 1], 128), ([400], [150], 64), ([400], [150], 128), ([900], [200], 256)])
@pytest.mark.parametrize("cap", [600.0, 1e4, 1e6, 3e38])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_cap_far_above_the_scores(kv, new, dim, cap, dtype):
    """A cap that hardly bends a score takes nothing from its accuracy: c tanh(s / c) to 2^-20 of s where s < c / 8 (the
    quotient and the product round by 2^-24 each, three terms and their factors by 2^-23 together, and the next term
    of the series that starts x - x^3 / 3 is far below), in place of a part of c."""
    cache, table, refs = build(kv, 2, dim, 16, "Q8_0", "Q8_0", 14)
    q = torch.randn(sum(new), 4, dim, generator=torch.Generator().manual_seed(4)).to(TYPES[dtype])
    start = np.concatenate([[0], np.cumsum(new)])
    out = ft.attn_kv(cache, q.cuda(), table, ints(kv), ints(start), softcap=cap).double().cpu().numpy()
    for i, (n, c) in enumerate(zip(kv, new)):
        a = slice(start[i], start[i + 1])
        o, terms, bias, mass = kv_ref.attention(q[a].double().numpy(), *refs[i], c, n, softcap=cap)
        # the bound's terms grow with the sum of |q k|, which is at least the score: 16 more units of 2^-24 of it
        bound = kv_ref.attention_bound(o, terms * (71 / 55), bias, mass, refs[i][1], dtype)
        assert np.all(np.abs(out[a] - o) <= bound), np.max(np.abs(out[a] - o) / bound)
