"""GPU: rows, pages and adapters that lie beyond 2^32 bytes and 2^31 elements from their base."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import layer_ref as ref
from tests.gpu_util import dev, host, need_gpu
from tests.test_gpu_lora import check as check_lora
from tests.test_gpu_norm import check as check_norm, vector
from tests.test_gpu_rope import check as check_rope, setup

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 8   # elements between rows


def far_rows(rows, width, seed):
    """(rows, width) bf16, rows FAR elements apart."""
    base = torch.empty((rows - 1) * FAR + width, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((rows, width), (FAR, 1))
    x.copy_(torch.randn(rows, width, generator=torch.Generator().manual_seed(seed)).cuda())
    return x


def test_rope_and_norm():
    need_gpu()
    x = far_rows(3, 256, 1)
    pos, tab = setup(3, 128)
    rows = x.unflatten(1, (2, 128))
    near = ft.rope(rows, dev(pos), dev(tab))
    check_rope(near, rows, pos, tab, False, "bf16")
    w = vector(256, 2)
    r, n, _ = ft.norm(x, weight=dev(w), residual=x, scale=0.5)
    check_norm((r, n), x, "bf16", residual=x, scale=0.5, weight=w)
    assert ft.rope(rows, dev(pos), dev(tab), out=rows) is rows   # written there too
    assert torch.equal(rows, near)


def test_store():
    need_gpu()
    page, heads, dim = 256, 8, 256
    n_pages = 2 ** 32 // ft.kv_page_bytes("Q8_0", page, heads, dim) + 20
    cache = ft.KvCache.empty(n_pages, page, heads, dim)
    g = torch.Generator().manual_seed(3)
    slots = torch.cat([torch.tensor([5, n_pages * page - 1]), (n_pages - 3) * page + torch.arange(40)]).cuda()
    t = slots.numel()
    k, v = (torch.randn(t, heads, dim, generator=g).cuda() for _ in range(2))
    pos, tab = setup(t, dim)
    ft.kv_store_rope(cache, None, k, v, slots, dev(pos), dev(tab))
    near = ft.KvCache.empty(2, page, heads, dim)
    to = torch.arange(t).cuda()
    ft.kv_store(near, ft.rope(k, dev(pos), dev(tab)), v, to)
    for a, b in zip(ft.kv_load(cache, slots), ft.kv_load(near, to)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("t", [3, 70])
def test_adapters(t):
    need_gpu()
    many, rank, k, n = 2049, 256, 4100, 4100   # 2.15 G elements each
    a, b = (torch.empty(many, *s, dtype=torch.bfloat16, device="cuda") for s in ((rank, k), (n, rank)))
    g = torch.Generator().manual_seed(4)
    for i in (0, many - 1):
        a[i].copy_(torch.randn(rank, k, generator=g).cuda() * k ** -0.5)
        b[i].copy_(torch.randn(n, rank, generator=g).cuda() * rank ** -0.5)
    x = torch.randn(t, k, generator=g).cuda()
    ids = torch.where(torch.arange(t) % 3 == 1, 0, many - 1).int().cuda()
    out = ft.lora(x, a, b, ids)
    some = torch.cat([a[:1], a[-1:]]), torch.cat([b[:1], b[-1:]])
    check_lora(out, x, *some, (ids > 0).int())
