"""GPU: the scored router where its fp32 order is at its limits."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_route_ex import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("e,n_group,topk_group,topk", [(64, 8, 2, 8), (256, 8, 4, 8), (160, 8, 3, 6), (36, 3, 2, 7), (512, 16, 5, 4),
                                                       (1024, 64, 9, 8), (128, 32, 1, 2)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("t", [60, 2050])
def test_groups_that_fp32_cannot_tell_apart(e, n_group, topk_group, topk, group_top, t):
    """Every group's best logit one of a few neighbouring numbers, of which many have the same sigmoid in fp32: in 64 bits
    the groups are in order, and no more than topk_group of them are open."""
    g = torch.Generator().manual_seed(e + n_group)
    x = -1 - torch.rand(t, n_group, e // n_group, generator=g)
    best = 2 + torch.rand(t, 1, generator=g) + torch.randint(0, 2 * n_group, (t, n_group), generator=g) * 2.0 ** -22
    x.scatter_(2, torch.randint(0, e // n_group, (t, n_group, 1), generator=g), best.unsqueeze(-1))
    kw = dict(score="sigmoid", n_group=n_group, topk_group=topk_group, group_top=group_top)
    check(x.flatten(1), topk, **kw)
    if t > 60:
        return
    check(x.flatten(1), topk, bias=torch.zeros(e), **kw)
    check(x.flatten(1) + 4, topk, renorm=False, **kw)


def test_groups_of_a_prompt():
    """Drawn logits, where a border between groups that close is one in thousands."""
    for seed in range(3):
        x = 1.5 * torch.randn(6000, 64, generator=torch.Generator().manual_seed(64 + seed))
        check(x, 8, score="sigmoid", n_group=8, topk_group=2)
        check(x, 6, score="sigmoid", n_group=16, topk_group=4, group_top=2, bias=torch.zeros(64))


@pytest.mark.parametrize("e", [40, 128, 256, 400, 1000])
@pytest.mark.parametrize("t", [50, 2100])
def test_scores_far_below_the_bias(e, t):
    """Scores under 1e-7 of the choice: the bias decides up to its own last bits, the scores below them."""
    g = torch.Generator().manual_seed(e)
    x = -17 + 0.3 * torch.randn(t, e, generator=g)
    near = 1 + torch.randint(0, 6, (e,), generator=g) * 2.0 ** -23       # biases a few last bits apart
    check(x, 8, score="sigmoid", bias=near)
    if t > 50:
        return
    check(x - 4, 8, score="sigmoid", bias=near)
    check(x, 8, score="sigmoid", bias=(1 + 2.0 ** -20 * torch.rand(e, generator=g)))
    if e % 4 == 0:
        check(x, 8, score="sigmoid", bias=near, n_group=4, topk_group=2, group_top=2)


@pytest.mark.parametrize("t", [7, 2100])
@pytest.mark.parametrize("e,topk,kw", [(8, 8, {}), (30, 30, {}), (32, 32, {}), (128, 8, dict(n_group=16, topk_group=1)),
                                       (64, 16, dict(n_group=8, topk_group=2)), (512, 16, dict(n_group=32, topk_group=1)),
                                       (1000, 25, dict(n_group=40, topk_group=1, group_top=2))])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_every_open_expert_is_chosen(e, topk, kw, t, score):
    g = torch.Generator().manual_seed(e + t)
    x = 1.5 * torch.randn(t, e, generator=g)
    check(x, topk, score=score, **kw)
    check(x.bfloat16(), topk, score=score, bias=0.1 * torch.randn(e, generator=g), **kw)
