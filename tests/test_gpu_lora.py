"""GPU: low-rank adapters against their definition in 64 bits, within the roundings of fp32 sums."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import layer_ref as ref
from tests.gpu_util import dev, host, need_gpu, own_stream
from tests.test_gpu_host_threads import together

pytestmark = pytest.mark.gpu


def case(t, k, n, many, rank, tx="f32", tw="bf16", seed=1, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, k + pad, generator=g).to(ref.DT[tx]).cuda()[:, :k]
    a = torch.randn(many, rank, k, generator=g).to(ref.DT[tw]).cuda()
    b = torch.randn(many, n, rank, generator=g).to(ref.DT[tw]).cuda()
    y = torch.randn(t, n + pad, generator=g).cuda()[:, :n]
    ids = torch.randint(-1, many + 1, (t,), generator=g, dtype=torch.int32).cuda()
    ids[0] = min(1, many - 1)
    return x, a, b, y, ids, torch.linspace(0.5, 2.0, many).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(out, x, a, b, ids, y=None, scales=None, ranks=None, rows=None):
    r, bound = ref.lora(f64(x), f64(a), f64(b), host(ids), f64(y), f64(scales), None if ranks is None else host(ranks))
    o = f64(out)
    if rows is not None:
        o, r, bound = o[rows], r[rows], bound[rows]
    off = np.abs(o - r)
    assert np.all(off <= bound + 1e-30), (np.max(off / (bound + 1e-30)), np.unravel_index(np.argmax(off / (bound + 1e-30)), off.shape))


@pytest.mark.parametrize("tx", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tw", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k,n,rank", [(64, 96, 16), (40, 77, 8), (7, 5, 3), (130, 300, 20), (1, 1, 1), (96, 256, 64), (33, 260, 100)])
def test_types_and_sizes(k, n, rank, tx, tw):
    """Short axes: the bound would show a piece of an operand left out."""
    need_gpu()
    for t in (1, 5, 17, 64, 100):
        x, a, b, y, ids, sc = case(t, k, n, 3, rank, tx, tw, seed=t)
        check(ft.lora(x, a, b, ids, y=y, scales=sc), x, a, b, ids, y, sc)


@pytest.mark.parametrize("t,many", [(1, 1), (2, 2), (16, 1), (17, 1), (31, 2), (33, 1), (48, 1), (49, 1), (63, 1), (64, 1), (64, 64), (65, 1), (65, 64), (127, 1),
                                    (128, 3), (129, 1), (300, 40), (1000, 7), (1100, 1), (2500, 300), (130, 8192), (40, 2000), (64, 1023), (64, 1024), (64, 1025), (200, 200)])
def test_tiles(t, many):
    """Every number of groups of tokens, and of adapters beside them."""
    need_gpu()
    for tx, tw in (("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")):
        x, a, b, y, ids, sc = case(t, 72, 40, many, 8, tx, tw, seed=t + many)
        check(ft.lora(x, a, b, ids, y=y, scales=sc), x, a, b, ids, y, sc)


@pytest.mark.parametrize("k,n,rank,t", [(4096, 600, 16, 3), (4096, 600, 16, 90), (1536, 2048, 64, 40), (14336, 130, 32, 20), (5000, 100, 128, 70),
                                        (2049, 515, 256, 10), (600, 300, 200, 150), (4100, 64, 8, 700)])
def test_long_axes(k, n, rank, t):
    """The long axis in shares, ranks past one workgroup's."""
    need_gpu()
    for tx, tw in (("f32", "f16"), ("bf16", "bf16")):
        x, a, b, y, ids, sc = case(t, k, n, 4, rank, tx, tw, seed=k)
        check(ft.lora(x, a, b, ids, y=y, scales=sc), x, a, b, ids, y, sc)


@pytest.mark.parametrize("t", [6, 80])
def test_ranks_of_their_own(t):
    """What lies beyond an adapter's rank is not used, whatever it is; a rank of 0 adds nothing, one too large counts as all."""
    need_gpu()
    for tx, tw, rank in (("f32", "bf16", 64), ("f16", "f16", 24), ("f32", "f32", 9)):
        x, a, b, y, ids, sc = case(t, 160, 90, 6, rank, tx, tw)
        ranks = torch.tensor([rank, 5, 0, 1, -3, rank + 100], dtype=torch.int32, device="cuda")
        ids = (torch.arange(t, dtype=torch.int32, device="cuda") * 5 + 1) % 7
        for i, r in enumerate(ranks.tolist()):
            a[i, max(0, r):] = float("nan")
            b[i, :, max(0, r):] = float("inf")
        check(ft.lora(x, a, b, ids, y=y, scales=sc, ranks=ranks), x, a, b, ids, y, sc, ranks)


@pytest.mark.parametrize("t", [5, 70])
def test_rows_without_an_adapter(t):
    need_gpu()
    x, a, b, y, ids, sc = case(t, 64, 530, 2, 16)
    ids[:] = torch.tensor([-1, 2, 0, -2 ** 31, 2 ** 31 - 1] * (t // 5), dtype=torch.int32)
    out = ft.lora(x, a, b, ids, y=y, scales=sc)
    check(out, x, a, b, ids, y, sc)
    none = (ids < 0) | (ids >= 2)
    assert torch.equal(out[none], y[none])
    out = ft.lora(x, a, b, ids, scales=sc)
    assert torch.all(out[none] == 0)
    check(out, x, a, b, ids, None, sc)
    ids[:] = -1
    assert torch.equal(ft.lora(x, a, b, ids, y=y), y)


@pytest.mark.parametrize("pad", [0, 1, 4, 8])
@pytest.mark.parametrize("t", [7, 75])
def test_strides_and_in_place(t, pad):
    need_gpu()
    for tx in ("f32", "bf16"):
        x, a, b, y, ids, sc = case(t, 104, 130, 3, 16, tx, pad=pad)
        want = ft.lora(x, a, b, ids, y=y, scales=sc)
        check(want, x, a, b, ids, y, sc)
        wide = torch.full((t, 130 + 2 * pad + 2), 7.0, device="cuda")
        out = ft.lora(x, a, b, ids, y=y, scales=sc, out=wide[:, pad:pad + 130])
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert torch.all(wide == 7.0)
        assert ft.lora(x, a, b, ids, y=y, scales=sc, out=y) is y
        assert torch.equal(y, want)


@pytest.mark.parametrize("t", [4, 40, 90])
def test_rows_keep_to_themselves(t):
    need_gpu()
    x, a, b, y, ids, sc = case(t, 256, 100, 2, 16)
    ids[:] = 1
    want = ft.lora(x, a, b, ids, y=y).clone()
    x[2, 5], x[3, 200] = float("nan"), float("-inf")
    out = ft.lora(x, a, b, ids, y=y)
    keep = torch.tensor([i for i in range(t) if i not in (2, 3)], device="cuda")
    assert torch.equal(out[keep], want[keep])
    assert torch.isnan(out[2:4]).all()
    x[2:4] = 1e38   # large, and finite in pieces
    check(ft.lora(x, a * 1e-3, b * 1e-3, ids, y=y), x, a * 1e-3, b * 1e-3, ids, y, rows=keep.cpu().numpy())


@pytest.mark.parametrize("tx,tw", [("f16", "f16"), ("f16", "bf16"), ("bf16", "bf16"), ("f32", "f16"), ("f32", "f32")])
def test_small_and_large_values(tx, tw):
    """Values down to a type's least, and up to where only the product is finite."""
    need_gpu()
    for t in (3, 70):
        for sx, sw in ((2.0 ** -24, 1.0), (2.0 ** -20, 2.0 ** -20), (2.0 ** 14, 2.0 ** -14), (2.0 ** -14, 2.0 ** 10)):
            x, a, b, y, ids, sc = case(t, 48, 50, 2, 8)
            x, a, b = ((v * s).to(ref.DT[d]) for v, s, d in ((x, sx, tx), (a, sw, tw), (b, 1.0, tw)))
            check(ft.lora(x, a, b, ids), x, a, b, ids)


def test_nothing_to_do():
    need_gpu()
    x, a, b, y, ids, sc = case(3, 16, 8, 2, 4)
    assert ft.lora(x[:0], a, b, ids[:0]).shape == (0, 8)
    assert ft.lora(x, a, b[:, :0].contiguous(), ids).shape == (3, 0)


@pytest.mark.parametrize("t", [9, 200])
def test_two_graphs_with_workspaces(t):
    """Captured on one stream, each with its own workspace; replayed with other ids and rows."""
    need_gpu()
    s, sets = own_stream(), []
    need = ft.lora_scratch_bytes(t, 1024, 5, 16)
    for i in range(2):
        x, a, b, y, ids, sc = case(t, 1024, 300, 5, 16, seed=60 + i)
        out, ws = torch.empty(t, 300, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            ft.lora(x, a, b, ids, y=y, scales=sc, out=out, workspace=ws, stream=s)
        sets.append((graph, x, a, b, ids, y, sc, out))
    for rep in range(3):
        for graph, x, a, b, ids, y, sc, out in sets:
            ids.copy_((ids + 1) % 5)
            x.mul_(-1.25)
        torch.cuda.synchronize()
        for graph, *_ in sets:
            graph.replay()
        torch.cuda.synchronize()
        for graph, x, a, b, ids, y, sc, out in sets:
            assert torch.equal(out, ft.lora(x, a, b, ids, y=y, scales=sc))
            check(out, x, a, b, ids, y, sc)


def test_capture_needs_scratch():
    need_gpu()
    x, a, b, y, ids, sc = case(9, 1024, 300, 5, 16)
    s, graph = own_stream(), torch.cuda.CUDAGraph()
    out = torch.zeros(9, 300, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(ft.FtError) as e:
            ft.lora(x, a, b, ids, y=y, out=out, stream=s)
        out.add_(0.0)
    assert ft.STATUS[e.value.status] == "FT_ERR_NO_SCRATCH"
    ft.scratch_reserve(ft.lora_scratch_bytes(9, 1024, 5, 16), stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ft.lora(x, a, b, ids, y=y, out=out, stream=s)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, a, b, ids, y)
    small = torch.empty(ft.lora_scratch_bytes(9, 1024, 5, 16) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(ft.FtError):
        ft.lora(x, a, b, ids, workspace=small)


def test_streams_and_threads():
    need_gpu()
    calls = []
    for seed in range(4):
        x, a, b, y, ids, sc = case(30 + 40 * seed, 512, 200, 4, 16, seed=seed)
        calls.append(lambda x=x, a=a, b=b, ids=ids, y=y: ft.lora(x, a, b, ids, y=y))
    together(calls)
    streams = [own_stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for s, (c, seed) in zip(streams, zip(calls, range(4))):
            with torch.cuda.stream(s):
                outs.append(c())
        torch.cuda.synchronize()
        for o, c in zip(outs, calls):
            assert torch.equal(o, c())
