"""GPU: rows stored and read back by workgroups of 4, 16 and 64 tokens (as the sizes decide), with runs of consecutive
slots that start anywhere, padding, and slots that stand alone between them: every byte of the pools against the plain form."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests import layer_ref as ref
from tests.gpu_util import dev, host, need_gpu

pytestmark = pytest.mark.gpu
SPANS = {4: (30, 4), 16: (200, 8), 64: (1300, 8)}   # tokens and heads


def span_of(t, heads):
    """Tokens per workgroup: csrc/ft_kv_store.h's rule for values that are read back."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    if -(-t // 4) * heads <= cus:
        return 4
    return 16 if -(-t // 16) * heads <= 2 * cus else 64


def places(ty, side, page, dim):
    """Byte and shift of every (token, element) of a page head: include/ft.h's layout."""
    j, e = np.arange(page)[:, None], np.arange(dim)[None, :]
    b, i, nb = e // 32, e % 32, dim // 32
    none = 0 * (j + e)
    if side == "v":
        return (e * page + j, none) if ty == "Q8_0" else ((16 * b + i % 16) * page + j, 4 * (i // 16) + none)
    if ty == "Q8_0":
        m = np.minimum(2, nb - b // 2 * 2)
        return page * 64 * (b // 2) + j * 32 * m + i // 8 * 8 * m + b % 2 * 8 + i % 8, none
    m = np.minimum(4, nb - b // 4 * 4)
    nibble = i % 8 // 2 + 4 * (i % 2)
    return page * 64 * (b // 4) + j * 16 * m + i // 8 * 4 * m + b % 4 * 4 + nibble // 2, 4 * (nibble % 2) + none


def written(before, x, ty, side, page, heads, dim, slots):
    """The pool's bytes with the rows x [t, heads, dim] in their slots."""
    pool = before.reshape(-1, heads, page * (dim // 32) * kv_ref.BLOCK_BYTES[ty]).copy()
    q, d = kv_ref.quantize(x, ty)
    q = np.where(np.repeat(d == 0, 32, -1), 0, q)
    at, shift = places(ty, side, page, dim)
    scales = kv_ref.code_bytes(ty, dim, page) + 2 * page * np.arange(dim // 32)
    for n, s in enumerate(slots):
        if s < 0 or s >= len(pool) * page:
            continue
        p, j = pool[s // page], s % page
        if ty == "Q8_0":
            p[:, at[j]] = (q[n] + 128).astype(np.uint8)
        else:
            p[:, at[j]] = 0                    # both nibbles of a byte are this token's
            for h in (0, 4):
                e = np.flatnonzero(shift[j] == h)
                p[:, at[j, e]] |= ((q[n][:, e] + 8) << h).astype(np.uint8)
        for k in range(2):
            p[:, scales + 2 * j + k] = d[n].view(np.uint8).reshape(heads, -1, 2)[..., k]
    return pool.reshape(before.shape)


def slots_of(t, start, page, seed):
    """Consecutive slots from `start` on in pages of any order, some of them padding, past the pool, or far from their neighbours."""
    rs = np.random.RandomState(seed)
    n_pages = (start + t) // page + 4
    order = rs.permutation(n_pages)
    j = np.arange(start, start + t)
    slots = order[j // page].astype(np.int64) * page + j % page
    spare = order[-2] * page + rs.permutation(page)          # a page of slots that stand alone
    lone = np.sort(rs.choice(t, min(t // 9 + 1, page), replace=False))
    slots[lone] = spare[:len(lone)]
    for n, s in zip(rs.choice(t, 4, replace=False), (-1, -5, n_pages * page, 1 << 40)):
        slots[n] = s
    return slots, n_pages


@pytest.mark.parametrize("k,v", [("Q8_0", "Q8_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0"), ("Q4_0", "Q4_0")])
@pytest.mark.parametrize("dim,page", [(64, 16), (96, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("span", SPANS)
def test_every_byte(span, dim, page, k, v):
    need_gpu()
    t, heads = SPANS[span]
    assert span_of(t, heads) == span
    rs = np.random.RandomState(dim + span)
    for start, turned in ((0, False), (7, False), (30, True), (16, True)):
        slots, n_pages = slots_of(t, start, page, start + t)
        dtype = {0: "f32", 7: "bf16", 30: "f32", 16: "f16"}[start]
        x, y = (torch.from_numpy(rs.standard_normal((t, heads, dim)).astype(np.float32)).to(ref.DT[dtype]) for _ in range(2))
        cache = ft.KvCache.empty(n_pages, page, heads, dim, k, v)
        cache.k_pages.copy_(torch.randint(0, 256, cache.k_pages.shape, dtype=torch.uint8))
        cache.v_pages.copy_(torch.randint(0, 256, cache.v_pages.shape, dtype=torch.uint8))
        before, ds = (host(cache.k_pages).copy(), host(cache.v_pages).copy()), dev(slots)
        keys = x.float().numpy()
        if turned:
            rot = dim // 2
            pos = rs.randint(0, 500, t).astype(np.int32)
            tab = ref.table(500, ft.rope_freqs(rot)[0]).astype(np.float32)
            keys = ref.turn(keys, pos, tab, False, kind=np.float32)
            q = torch.from_numpy(rs.standard_normal((t, 3, dim)).astype(np.float32)).to(ref.DT[dtype]).cuda()
            out = ft.kv_store_rope(cache, q, x.cuda(), y.cuda(), ds, dev(pos), dev(tab))
            assert torch.equal(out, ft.rope(q, dev(pos), dev(tab)))
        else:
            ft.kv_store(cache, x.cuda(), y.cuda(), ds)
        for pool, old, rows, ty, side in ((cache.k_pages, before[0], keys, k, "k"), (cache.v_pages, before[1], y.float().numpy(), v, "v")):
            same = np.array_equal(host(pool), written(old, rows, ty, side, page, heads, dim, slots))
            assert same, (start, side)
        there = torch.from_numpy((slots >= 0) & (slots < n_pages * page)).view(-1, 1, 1)
        for got, rows, ty in zip(ft.kv_load(cache, ds, dtype=ref.DT[dtype]), (keys, y.float().numpy()), (k, v)):
            want = torch.from_numpy(kv_ref.values(*kv_ref.quantize(rows, ty))).float().to(ref.DT[dtype])
            same = torch.equal(got.cpu(), torch.where(there, want, torch.zeros_like(want)))
            assert same, (start, ty)


def test_layout_of_the_plain_form():
    """The vectorised layout above is the one that is read element by element elsewhere."""
    rs = np.random.RandomState(1)
    for ty in ("Q8_0", "Q4_0"):
        for side in "kv":
            for dim, page in ((64, 16), (96, 32), (256, 16)):
                x = rs.standard_normal((3, 2, dim)).astype(np.float32)
                pool = np.zeros((2, 2 * page * (dim // 32) * kv_ref.BLOCK_BYTES[ty]), np.uint8)
                pool = written(pool, x, ty, side, page, 2, dim, [page + 3, 5, 0])
                q, d = kv_ref.quantize(x, ty)
                for n, s in enumerate((page + 3, 5, 0)):
                    gq, gd = kv_ref.read_slot(pool, ty, side, page, 2, dim, s)
                    assert np.array_equal(gq, q[n]) and np.array_equal(gd, d[n])
