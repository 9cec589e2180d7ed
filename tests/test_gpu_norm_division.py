"""GPU: the blocks of ft.norm against torch's own operations on the GPU, code by code and scale by scale.

Scales are amax / 127, an IEEE division.  torch divides by a tensor that way; a division by a number in the program, x / 127,
it computes on the GPU as a product with the rounded reciprocal, which moves the last bit of one scale in twenty, and with it
now and then the code of a value next to a half-integer."""
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BLOCK = {"Q8_1": (32, 36, 4), "Q8_0": (32, 34, 2), "Q8_K": (256, 292, 4)}   # elements, bytes, where the codes begin


def rms(x, eps):
    return x * (1.0 / (x.double().square().mean(-1, keepdim=True) + eps).sqrt()).float()


@pytest.mark.parametrize("act", BLOCK)
def test_codes_by_true_division(act):
    need_gpu()
    size, bytes_, first = BLOCK[act]
    eps = 1e-6
    for seed in range(40):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, residual = (torch.randn(37, 2048, generator=g, device="cuda") for _ in range(2))
        post, weight, gate = (1 + 0.1 * torch.randn(2048, generator=g, device="cuda") for _ in range(3))
        r, _, xq = ft.norm(x, weight=weight, post_weight=post, gate=gate, residual=residual, act=act, eps=eps)
        want = residual + rms(x, eps) * post * gate
        assert torch.equal(r, want), seed
        v = (rms(want, eps) * weight).unflatten(1, (-1, size))
        top = v.abs().amax(-1, keepdim=True)
        d = top / torch.full_like(top, 127.0)
        if act != "Q8_K":
            d = d.half()
        q = v / d.float()
        q = torch.copysign(torch.floor(q.double().abs() + 0.5), q).float().clamp(-127, 127)
        blocks = xq.view(37, -1, bytes_)
        codes = blocks[..., first:first + size].view(torch.int8).float()
        scales = blocks[..., :4].view(torch.float32) if act == "Q8_K" else blocks[..., :2].view(torch.float16)
        assert torch.equal(scales, d), seed
        assert torch.equal(codes, q), seed
