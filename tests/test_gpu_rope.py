"""GPU: rotary positions against their definition, and the store that turns its rows against the two calls it stands for."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import layer_ref as ref
from tests.gpu_util import dev, host, need_gpu, own_stream

pytestmark = pytest.mark.gpu


def rows(t, heads, dim, dtype, seed=1, pad=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(t, heads, dim + pad, generator=g).to(ref.DT[dtype]).cuda()[..., :dim]


def setup(t, rot, n_pos=300, seed=2):
    freqs, _ = ft.rope_freqs(rot, 1000.0)
    pos = np.random.RandomState(seed).randint(0, n_pos, t).astype(np.int32)
    tab = ref.table(n_pos, freqs).astype(np.float32)
    return pos, tab


def check(out, x, pos, tab, interleaved, dtype, weight=None, eps=0.0):
    f = x.double().cpu().numpy()
    r = ref.turn(f, pos, tab, interleaved, weight, eps)
    # two products, a sum (and two products and a factor of the norm), each off by half a step of its value
    i, j = ref.pairs(x.shape[-1], tab.shape[1], interleaved)
    c, s = (np.abs(tab[np.clip(pos, 0, len(tab) - 1)])[:, None, k * (tab.shape[1] // 2):(k + 1) * (tab.shape[1] // 2)] for k in (0, 1))
    flat = np.concatenate([np.ones_like(tab[:, :tab.shape[1] // 2]), np.zeros_like(tab[:, tab.shape[1] // 2:])], 1)
    v = np.abs(ref.turn(f, pos, flat, interleaved, weight, eps))   # normed, not turned
    terms = v.copy()
    terms[..., i], terms[..., j] = v[..., i] * c + v[..., j] * s, v[..., j] * c + v[..., i] * s
    bound = (2 if weight is None else 5) * 1.01 * 2.0 ** -24 * terms + ref.rounding(r, dtype) + 2.0 ** -40
    off = np.abs(out.double().cpu().numpy() - r)
    assert np.all(off <= bound), np.max(off / bound)
    if dtype == "f32":  # every rounding is fixed
        single = ref.turn(x.cpu().numpy(), pos, tab, interleaved, weight, eps, np.float32)
        assert np.array_equal(host(out), single)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 64), (64, 16), (96, 96), (80, 80), (80, 40), (192, 64), (256, 256), (2, 2), (10, 6),
                                     (33, 32), (12, 12), (512, 512), (100, 98), (64, 2)])
def test_turned_rows(dim, rot, interleaved, dtype):
    need_gpu()
    for t, heads, weighted in ((1, 1, False), (5, 3, True), (67, 2, False)):
        x = rows(t, heads, dim, dtype)
        pos, tab = setup(t, rot)
        w = (1 + 0.3 * np.random.RandomState(5).randn(dim)).astype(np.float32) if weighted else None
        out = ft.rope(x, dev(pos), dev(tab), interleaved=interleaved, weight=None if w is None else dev(w), eps=1e-5)
        check(out, x, pos, tab, interleaved, dtype, w, 1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (64, 24, False), (80, 80, True)])
def test_many_rows(dim, rot, interleaved, dtype):
    """Several heads per wave, the last group with fewer."""
    need_gpu()
    t, heads = 12000, 9
    x = rows(t, heads, dim, dtype)
    pos, tab = setup(t, rot)
    check(ft.rope(x, dev(pos), dev(tab), interleaved=interleaved), x, pos, tab, interleaved, dtype)


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(pad, interleaved):
    need_gpu()
    t, heads, dim, rot = 37, 5, 128, 96
    for dtype in ("f32", "bf16"):
        x = rows(t, heads, dim, dtype, pad=pad)
        pos, tab = setup(t, rot)
        wide = torch.full((t, heads + 2, dim + pad), 7.0, dtype=x.dtype, device="cuda")
        out = ft.rope(x, dev(pos), dev(tab), interleaved=interleaved, out=wide[:, 1:1 + heads, :dim])
        check(out, x, pos, tab, interleaved, dtype)
        out.fill_(7.0)
        assert torch.all(wide == 7.0)   # nothing beside the rows was written
        back = x.clone()
        assert ft.rope(back, dev(pos), dev(tab), interleaved=interleaved, out=back) is back
        check(back, x, pos, tab, interleaved, dtype)
        swapped = rows(heads, t, dim, dtype).transpose(0, 1)   # heads further apart than tokens
        check(ft.rope(swapped, dev(pos), dev(tab), interleaved=interleaved), swapped, pos, tab, interleaved, dtype)


def test_positions_outside_the_table():
    need_gpu()
    x = rows(6, 2, 64, "f32")
    pos, tab = np.array([-1, -2 ** 31, 299, 300, 2 ** 31 - 1, 0], np.int32), setup(1, 64)[1]
    check(ft.rope(x, dev(pos), dev(tab)), x, pos, tab, False, "f32")


def test_nothing_to_do_and_special_values():
    need_gpu()
    pos, tab = setup(0, 64)
    assert ft.rope(rows(0, 4, 64, "f32"), dev(pos), dev(tab)).shape == (0, 4, 64)
    pos, tab = setup(4, 32)
    x = rows(4, 3, 64, "f32")
    x[1, 1, 3], x[2, 0, 50] = float("nan"), float("inf")   # a pair's; an element that does not turn
    out = host(ft.rope(x, dev(pos), dev(tab)))
    bad = np.argwhere(~np.isfinite(out))
    assert sorted(map(tuple, bad)) == [(1, 1, 3), (1, 1, 19), (2, 0, 50)]
    assert out[2, 0, 50] == np.inf
    x = rows(2, 2, 64, "f32") * 1e25   # squares past fp32
    w = np.ones(64, np.float32)
    check(ft.rope(x, dev(pos[:2]), dev(tab), weight=dev(w)), x, pos[:2], tab, False, "f32", w)
    zero = torch.zeros(2, 2, 64, device="cuda")
    assert torch.all(ft.rope(zero, dev(pos[:2]), dev(tab), weight=dev(w), eps=1e-6) == 0)


@pytest.mark.parametrize("rot,n_pos,base", [(128, 5000, 10000.0), (2, 131072, 10000.0), (64, 40000, 500000.0)])
def test_table(rot, n_pos, base):
    need_gpu()
    freqs, scale = ft.rope_freqs(rot, base, "ramp", 4.0, 4096)
    got, want = host(ft.rope_table(n_pos, freqs, scale)).astype(np.float64), ref.table(n_pos, freqs, scale)
    assert got.shape == want.shape
    # rounded once; the angle itself is a 64-bit product, off by half a step of it
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) * 1.0001 + n_pos * 2.0 ** -52)
    assert ft.rope_table(0, freqs).shape == (0, rot)


def test_turned_back():
    """Negative angles are the inverse."""
    need_gpu()
    freqs, _ = ft.rope_freqs(128)
    x, pos = rows(9, 4, 128, "f32"), dev(np.arange(9, dtype=np.int32) * 777)
    there = ft.rope(x, pos, ft.rope_table(8000, freqs))
    back = ft.rope(there, pos, ft.rope_table(8000, [-f for f in freqs]))
    pair = torch.hypot(x[..., :64], x[..., 64:]).repeat(1, 1, 2)
    # each turn's cosine, sine, products and sum: 8 half steps of the pair's length, twice
    assert torch.all((back - x).abs() <= 16 * 2.0 ** -24 * pair)


# ---------------------------------------------------------------------------
# the store
# ---------------------------------------------------------------------------
def stored(cache):
    return cache.k_pages.clone(), cache.v_pages.clone()


def cleared(*shape):
    pools = [torch.full((shape[0], ft.kv_page_bytes(ty, *shape[1:4])), 0x5A, dtype=torch.uint8, device="cuda") for ty in shape[4:]]
    return ft.KvCache(*pools, *shape[1:])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("k,v", [("Q8_0", "Q8_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0"), ("Q4_0", "Q4_0")])
def test_store_is_turn_then_store(k, v, dim, dtype):
    need_gpu()
    hk, page, n_pages = 3, 16 if dim != 96 else 64, 40
    for t, heads, rot, interleaved, weighted in ((1, 6, dim, False, True), (70, 7, dim // 2, True, False), (133, 0, dim, False, True), (64, 1, 6, False, False)):
        fused = rows(t, heads + 2 * hk, dim, dtype, seed=t)
        q, kk, vv = fused[:, :heads], fused[:, heads:heads + hk], fused[:, heads + hk:]
        pos, tab = setup(t, rot)
        slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(t))[:t]
        if t > 2:
            slots[0], slots[1] = -1, n_pages * page   # neither is stored
        if t > 100:
            slots[40:80] = torch.arange(16 * 8, 16 * 8 + 40)   # a run over a page's end
            slots[:40] = -1
            slots[80:] = torch.arange(300, 300 + t - 80)
        slots = slots.cuda()
        w = [dev((1 + 0.3 * np.random.RandomState(i).randn(dim)).astype(np.float32)) if weighted else None for i in (5, 6)]
        got, want = (cleared(n_pages, page, hk, dim, k, v) for _ in range(2))
        out = ft.kv_store_rope(got, q if heads else None, kk, vv, slots, dev(pos), dev(tab), interleaved, w[0] if heads else None, w[1], 1e-5)
        turned = ft.rope(kk.float(), dev(pos), dev(tab), interleaved, w[1], 1e-5)
        ft.kv_store(want, turned, vv.float(), slots)
        for a, b in zip(stored(got), stored(want)):
            assert torch.equal(a, b)
        if heads:
            assert torch.equal(out, ft.rope(q, dev(pos), dev(tab), interleaved, w[0], 1e-5))
        else:
            assert out is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_store_of_a_prompt(dtype):
    """Several heads per wave; the queries in place."""
    need_gpu()
    t, heads, hk, dim, page = 8000, 13, 5, 128, 64
    fused = rows(t, heads + 2 * hk, dim, dtype)
    pos, tab = setup(t, dim)
    slots = torch.arange(t).flip(0).cuda()
    want_q = ft.rope(fused[:, :heads], dev(pos), dev(tab))
    got, want = (cleared(t // page, page, hk, dim, "Q8_0", "Q4_0") for _ in range(2))
    ft.kv_store(want, ft.rope(fused[:, heads:heads + hk].float(), dev(pos), dev(tab)), fused[:, heads + hk:].float(), slots)
    q = fused[:, :heads]
    ft.kv_store_rope(got, q, fused[:, heads:heads + hk], fused[:, heads + hk:], slots, dev(pos), dev(tab), q_out=q)
    assert torch.equal(fused[:, :heads], want_q)
    for a, b in zip(stored(got), stored(want)):
        assert torch.equal(a, b)


def test_captured():
    """A decode step in a graph, replayed with other contents."""
    need_gpu()
    t, heads, hk, dim, page = 4, 8, 2, 128, 16
    fused, (pos, tab) = rows(t, heads + 2 * hk, dim, "f32"), setup(t, dim)
    pos, tab, slots = dev(pos), dev(tab), torch.tensor([3, 40, 17, -1], device="cuda")
    cache, out = cleared(4, page, hk, dim, "Q8_0", "Q8_0"), torch.empty(t, heads, dim, device="cuda")
    s, graph = own_stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        ft.kv_store_rope(cache, fused[:, :heads], fused[:, heads:heads + hk], fused[:, heads + hk:], slots, pos, tab, q_out=out, stream=s)
        ft.rope(out, pos, tab, out=out, stream=s)
    for i in range(3):
        fused.copy_(rows(t, heads + 2 * hk, dim, "f32", seed=50 + i))
        pos.add_(1)
        slots.add_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        other = cleared(4, page, hk, dim, "Q8_0", "Q8_0")
        other.k_pages.copy_(cache.k_pages)
        other.v_pages.copy_(cache.v_pages)
        want = ft.kv_store_rope(other, fused[:, :heads], fused[:, heads:heads + hk], fused[:, heads + hk:], slots, pos, tab)
        assert torch.equal(out, ft.rope(want, pos, tab))
        assert all(torch.equal(a, b) for a, b in zip(stored(cache), stored(other)))
