"""GPU: rows quantized into the paged cache and read back, against the plain form."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import host, need_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def rows(t, heads, dim, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, heads, dim, generator=g) * torch.exp(2 * torch.randn(t, heads, 1, generator=g))
    if t > 2:
        x[1] = 0.0                                       # a zero row
        x[2, :, :32] = 2.0 ** -30 * x[2, :, :32]         # a scale that is subnormal in fp16, or zero
        x[2, :, 32:40] = 1.0                             # equal magnitudes of both signs: the first counts
        x[2, :, 40:48] = -1.0
        x[2, :, 48:64] = 0.5
    return x.to(dtype)


def check(cache, k, v, slots, heads, dim, page):
    """Every written slot holds the plain form's codes and scales, byte by byte."""
    kp, vp = host(cache.k_pages), host(cache.v_pages)
    for x, ty, side, pool in ((k, cache.k, "k", kp), (v, cache.v, "v", vp)):
        q, d = kv_ref.quantize(x.float().cpu().numpy(), ty)
        for i, s in enumerate(slots):
            if s < 0 or s >= cache.n_pages * page:
                continue
            gq, gd = kv_ref.read_slot(pool, ty, side, page, heads, dim, s)
            assert np.array_equal(gd.view(np.uint16), d[i].view(np.uint16)), (side, i, "scales")
            live = np.repeat(d[i] != 0, 32, -1)
            assert np.array_equal(gq[live], q[i][live]), (side, i, "codes")
            assert not gq[~live].any()


@pytest.mark.parametrize("k,v", [("Q8_0", "Q8_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0"), ("Q4_0", "Q4_0")])
@pytest.mark.parametrize("dim,page", [(64, 16), (96, 32), (128, 64), (256, 128), (128, 256)])
def test_store_bits(k, v, dim, page):
    heads, t = 3, 7
    cache = ft.KvCache.empty(3, page, heads, dim, k, v)
    cache.k_pages.fill_(0xA5)
    cache.v_pages.fill_(0x5A)
    before = host(cache.k_pages).copy(), host(cache.v_pages).copy()
    x, y = rows(t, heads, dim, 1, torch.float32), rows(t, heads, dim, 2, torch.float32)
    slots = [page + 3, 0, 2 * page + page - 1, -1, page + 4, 3 * page, 5]   # padding, and one past the pool
    ft.kv_store(cache, x.cuda(), y.cuda(), torch.tensor(slots).cuda())
    check(cache, x, y, slots, heads, dim, page)
    # nothing but the written slots changed
    for side, ty, pool, old in (("k", k, cache.k_pages, before[0]), ("v", v, cache.v_pages, before[1])):
        new = host(pool)
        for s in range(3 * page):
            if s not in slots and (s < 8 or s % page > page - 3):
                for a, b in zip(kv_ref.read_slot(new, ty, side, page, heads, dim, s),
                                kv_ref.read_slot(old, ty, side, page, heads, dim, s)):
                    assert np.array_equal(a.view(np.uint8), b.view(np.uint8)), (side, s)


@pytest.mark.parametrize("k,v", [("Q8_0", "Q4_0"), ("Q4_0", "Q8_0")])
@pytest.mark.parametrize("t,start", [(1, 0), (16, 0), (15, 16), (64, 32), (65, 7), (130, 30), (200, 16)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_runs_and_round_trip(k, v, t, start, dtype):
    """Consecutive slots that start anywhere (the 16-byte rows of V and the single bytes at the ends), pages in
    any order, and what comes back."""
    heads, dim, page = 2, 128, 32
    n_pages = (start + t) // page + 2
    cache = ft.KvCache.empty(n_pages, page, heads, dim, k, v)
    cache.k_pages.zero_()
    cache.v_pages.zero_()
    order = np.random.default_rng(t + start).permutation(n_pages)
    j = np.arange(start, start + t)
    slots = order[j // page] * page + j % page
    x, y = rows(t, heads, dim, 3, TYPES[dtype]), rows(t, heads, dim, 4, TYPES[dtype])
    ds = torch.from_numpy(slots).cuda()
    ft.kv_store(cache, x.cuda(), y.cuda(), ds)
    some = list(range(0, t, 17)) + [t - 1]
    check(cache, x[some], y[some], slots[some], heads, dim, page)
    for out in TYPES.values():
        gk, gv = ft.kv_load(cache, ds, dtype=out)
        for got, src, ty in ((gk, x, k), (gv, y, v)):
            q, d = kv_ref.quantize(src.float().numpy(), ty)
            want = torch.from_numpy(kv_ref.values(q, d)).float().to(out)   # d * q is exact in fp32
            assert torch.equal(got.cpu(), want), (out, ty)


def test_strided_rows_and_single_sides():
    """Columns of a fused product as input, a head-major output, unaligned rows, one side alone."""
    heads, dim, page, t = 4, 64, 16, 21
    cache = ft.KvCache.empty(4, page, heads, dim, "Q4_0", "Q8_0")
    fused = torch.randn(t, 5 + 2 * heads * dim, device="cuda")
    k = fused[:, 5:5 + heads * dim].unflatten(1, (heads, dim))
    v = fused[:, 5 + heads * dim:].unflatten(1, (heads, dim))
    slots = torch.arange(t, device="cuda") + 9
    ft.kv_store(cache, k, v, slots)
    ks, vs = ft.kv_load(cache, slots)
    out = torch.full((heads, t, dim), 7.0, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    _, v16 = ft.kv_load(cache, slots, k=torch.empty(t, heads, dim, device="cuda", dtype=torch.bfloat16), v=out)
    assert torch.equal(v16, vs.bfloat16())
    for got, src, ty in ((ks, k, "Q4_0"), (vs, v, "Q8_0")):
        assert np.array_equal(host(got), kv_ref.values(*kv_ref.quantize(host(src), ty)).astype(np.float32))
    # one side alone, through the library's own entry point
    one = torch.full((t, heads, dim), -1.0, device="cuda")
    st = ft.lib().ft_kv_load(cache._ref, slots.data_ptr(), t, 0, None, 0, 0, one.data_ptr(), heads * dim, dim,
                             torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(one, vs)


def test_padding_reads_zeros():
    cache = ft.KvCache.empty(2, 16, 1, 64)
    x = torch.randn(4, 1, 64, device="cuda")
    ft.kv_store(cache, x, x, torch.tensor([3, 4, 5, 6], device="cuda"))
    k, v = ft.kv_load(cache, torch.tensor([-1, 3, 32, 1 << 40], device="cuda"))
    for y in (k, v):
        assert not y[0].any() and y[1].any() and not y[2:].any()


def test_far_values():
    """Scales at the ends of fp16: the largest finite one, and blocks whose scale rounds to zero."""
    cache = ft.KvCache.empty(1, 16, 1, 64, "Q8_0", "Q4_0")
    x = torch.zeros(5, 1, 64)
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2], x[3, 0, 3], x[4, 0, 4] = 3e38, -3e38, 1e-30, 127 * 2.0 ** -24, -8 * 2.0 ** -24
    ft.kv_store(cache, x.cuda(), x.cuda(), torch.arange(5).cuda())
    check(cache, x, x, list(range(5)), 1, 64, 16)
    assert torch.isfinite(ft.kv_load(cache, torch.arange(5).cuda())[0]).all()
