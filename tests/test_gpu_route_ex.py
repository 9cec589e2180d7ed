"""GPU: the router with scores, bias and groups against its plain 64-bit form.

Weights: fp64 sums and exponentials, one rounding to fp32 (2^-24), and the few fp64
roundings below it: 2^-23 relative."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def check(x, topk, **kw):
    ids, w = ft.moe_route_ex(x.cuda(), topk, **{k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()})
    ref = dict(kw)
    ref["sigmoid"] = ref.pop("score", "softmax") == "sigmoid"
    if torch.is_tensor(ref.get("bias")):
        ref["bias"] = ref["bias"].numpy()
    ri, rw = kv_ref.route(x.float().numpy(), topk, **ref)
    assert np.array_equal(host(ids), ri)
    got = host(w).astype(np.float64)
    assert np.all(np.abs(got - rw) <= 2.0 ** -23 * np.abs(rw) + 1e-44)
    return ids, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (3, 8, 8), (5, 64, 6), (9, 65, 4), (4, 127, 8), (33, 128, 8), (7, 256, 8), (6, 384, 10),
                                      (2, 1024, 32), (3, 1000, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_plain(score, t, e, topk, dtype):
    g = torch.Generator().manual_seed(t * e)
    x = (2 * torch.randn(t, e, generator=g)).to(dtype)
    check(x, topk, score=score)
    check(x, topk, score=score, renorm=False, scale=2.5, bias=0.2 * torch.randn(e, generator=g))


@pytest.mark.parametrize("e,n_group,topk_group,topk", [(256, 8, 4, 8), (64, 64, 5, 5), (160, 8, 3, 6), (96, 2, 1, 8), (1024, 4, 2, 16),
                                                       (36, 3, 2, 7), (8, 4, 1, 2), (250, 10, 10, 8), (128, 16, 1, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(e, n_group, topk_group, topk, group_top, score):
    g = torch.Generator().manual_seed(e + n_group)
    x = 1.5 * torch.randn(19, e, generator=g)
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    check(x, topk, **kw)
    check(x, topk, bias=0.1 * torch.randn(e, generator=g), **kw)


def test_ties_and_closed_experts():
    x = torch.zeros(6, 40)
    x[1, 7] = x[1, 39] = 1.0
    x[2] = -float("inf")
    x[2, 3] = 2.0                                     # one expert open: the others have score 0
    x[3, ::2] = -float("inf")
    x[4] = torch.tensor([90.0, 91.0] * 20)            # sigmoid is 1 for both: a tie
    x[5, 20] = -0.0
    for score in ("softmax", "sigmoid"):
        check(x, 8, score=score)
        check(x, 4, score=score, n_group=4, topk_group=2, group_top=2, bias=torch.zeros(40))
    # nothing open at all: the first experts, weights 0 (softmax has no sum to divide by)
    ids, w = ft.moe_route_ex(torch.full((1, 8), -float("inf")).cuda(), 3)
    assert host(ids).tolist() == [[0, 1, 2]] and not host(w).any()


def test_nan_is_never_preferred():
    x = torch.randn(4, 96)
    x[:, 5] = float("nan")
    ids, _ = ft.moe_route_ex(x.cuda(), 8, score="sigmoid", n_group=3, topk_group=2)
    got = host(ids)
    assert (got != 5).all() and (got >= 0).all() and (got < 96).all()


def test_neighbours():
    """Scores a last bit apart, or equal, in an order that fp32 could not keep."""
    g = torch.Generator().manual_seed(5)
    x = 1 + torch.randint(0, 40, (64, 200), generator=g) * 2.0 ** -23
    bias = torch.randint(-2, 3, (200,), generator=g) * 2.0 ** -26
    for score in ("softmax", "sigmoid"):
        check(x, 16, score=score)
        check(x, 16, score=score, bias=bias)


@pytest.mark.parametrize("t", [5, 2049])
@pytest.mark.parametrize("e,topk", [(40, 15), (64, 32), (256, 15), (256, 32), (300, 30), (512, 31), (1000, 32)])
def test_many_slots_and_equal_logits(t, e, topk):
    """16-bit logits, of which many are equal, the last slot's and the first left out's among them."""
    g = torch.Generator().manual_seed(e + topk)
    for dtype, size in ((torch.bfloat16, 1.0), (torch.float16, 1.0), (torch.bfloat16, 0.02), (torch.bfloat16, 30.0)):
        x = (size * torch.randn(t, e, generator=g)).to(dtype)
        check(x, topk, score="sigmoid")
        check(x, topk, renorm=False)
    x = torch.randint(0, 6, (t, e), generator=g).to(torch.bfloat16)       # a few values only
    check(x, topk)
    check(x, topk, score="sigmoid", bias=(torch.randint(0, 3, (e,), generator=g) / 4).float())


def test_many_from_one_lane():
    """The best experts side by side: one lane of the kernel gives up all of its own, more than once."""
    for e, first in ((256, 0), (256, 64), (512, 128), (1024, 256), (64, 0), (128, 4)):
        x = torch.randn(2100, e, generator=torch.Generator().manual_seed(e + first)) * 0.1
        for i in range(12):                            # quads 64 (128, 256) apart are one lane's
            at = (first + i // 4 * (64 if e <= 256 else 128 if e <= 512 else 256) + i % 4) % e
            x[:, at] += 5 + i
        check(x[:40], 10)
        check(x, 10, score="sigmoid", bias=torch.zeros(e))
    x = -torch.arange(256.0).repeat(3000, 1)           # expert 0 first, its lane's others next
    check(x, 14)


def test_strided_rows_and_outputs():
    x = torch.randn(10, 300)
    wide = x.cuda()
    rows = wide[:, 17:17 + 128]
    ids = torch.empty(10, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(10, 8, device="cuda")
    a, b = ft.moe_route_ex(rows, 8, ids=ids, w=w)
    assert a is ids and b is w
    ri, rw = kv_ref.route(x[:, 17:17 + 128].numpy(), 8)
    assert np.array_equal(host(ids), ri)
    with pytest.raises(ValueError):
        ft.moe_route_ex(wide.t(), 8)
    with pytest.raises(ValueError):
        ft.moe_route_ex(rows, 8, ids=ids.long())
    with pytest.raises(ft.FtError):
        ft.moe_route_ex(rows, 8, n_group=3)


def test_agrees_with_the_plain_router():
    """Softmax over all experts, renormalised, is the softmax over the chosen ones."""
    x = torch.randn(50, 128, device="cuda")
    ids, w = ft.moe_route(x, 8)
    ids2, w2 = ft.moe_route_ex(x, 8)
    assert torch.equal(ids, ids2)
    assert (w - w2).abs().max().item() < 1e-6
