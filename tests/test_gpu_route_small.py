"""GPU: the scored router's weights where they are small against fp32's range, or below it."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import dev, host, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm,scale", [(True, 2.0), (False, 1.0)])
def test_weights_below_fp32(score, renorm, scale):
    """Within 2^-23 of itself or half of fp32's least number, 2^-150, whichever is more.  The bias chooses experts of any score; a
    weight is its score over the chosen ones' sum, which one score near 1 holds above 1/2."""
    need_gpu()
    t, e, topk = 64, 32, 6
    rs = np.random.RandomState(5)
    logits = np.float32(-rs.uniform(0, 130, (t, e)))
    logits[:, 3] = 4.0
    logits[::5, 7] = -800.0                       # e^-800 is no number of fp32, and e^-104 is less than half of the least
    logits[1::5, 9] = -104.5
    logits[2::5, 11] = -103.2
    bias = np.float32(rs.uniform(0, 1, e))
    bias[[3, 7, 9, 11]] = 3.0
    ids, w = ft.moe_route_ex(dev(logits), topk, score=score, bias=dev(bias), renorm=renorm, scale=scale)
    rid, rw = kv_ref.route(logits, topk, sigmoid=score == "sigmoid", bias=bias, renorm=renorm, scale=scale)
    assert np.array_equal(host(ids), rid)
    small = rw < 2.0 ** -126
    assert small.any() and (rw < 2.0 ** -150).any() and not small.all()
    off = np.abs(host(w).astype(np.float64) - rw)
    bound = np.maximum(2.0 ** -23 * rw, 2.0 ** -150 * 1.0001)
    assert np.all(off <= bound), np.max(off / bound)
