"""GPU: attention whose keys are split over workgroups: parts that hold no key, more parts than a wave joins at once,
captured calls whose lengths grow over the borders of the parts."""
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


def right(out, q, kv, new, refs, dtype, **kw):
    out, q = out.double().cpu().numpy(), q.double().cpu().numpy()
    start = np.concatenate([[0], np.cumsum(new)])
    for i, (n, c) in enumerate(zip(kv, new)):
        a = slice(start[i], start[i + 1])
        o, terms, bias, mass = kv_ref.attention(q[a], refs[i][0][:n], refs[i][1][:n], c, n, **kw)
        bound = kv_ref.attention_bound(o, terms, bias, mass, refs[i][1][:n], dtype)
        assert np.all(np.isfinite(out[a])) and np.all(np.abs(out[a] - o) <= bound), (i, n)


def wide(table, cols):
    t = torch.zeros(table.shape[0], cols, dtype=torch.int32, device="cuda")
    t[:, :table.shape[1]] = table
    return t


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("kv,new,max_kv", [([200], [150], 20000), ([90, 1, 200], [90, 1, 60], 9000), ([70], [3], 30000), ([0, 64], [1, 1], 30000)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_parts_without_keys(kv, new, max_kv, dim, dtype):
    """A host bound far above the lengths: most workgroups have nothing to do and say so."""
    cache, table, refs = build(kv, 2, dim, 16, "Q8_0", "Q8_0", 21)
    q = torch.randn(sum(new), 8, dim, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    args = (cache, q.cuda(), wide(table, -(-max_kv // 16)), ints(kv), ints(np.concatenate([[0], np.cumsum(new)])))
    assert ft.attn_kv_scratch_bytes(cache, sum(new), 8, len(new), max_kv) > 0
    right(ft.attn_kv(*args, max_kv=max_kv), q, kv, new, refs, dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_more_parts_than_a_wave_joins_at_once(dtype):
    """One key/value head of 70000 keys: 1095 steps of 64, 16 to a part, 69 parts (the join takes 64 at a time); a
    row whose largest score lies in the last part, one whose lies in the first."""
    n, dim, page = 70000, 64, 256
    g = torch.Generator().manual_seed(31)
    cache = ft.KvCache.empty(-(-n // page), page, 1, dim, "Q8_0", "Q8_0")
    x, y = torch.randn(2, n, 1, dim, generator=g)
    q = torch.randn(1, 4, dim, generator=g).to(TYPES[dtype])
    x[-3, 0] = 3 * q[0, 0].float()
    x[5, 0] = 3 * q[0, 1].float()
    ft.kv_store(cache, x.cuda(), y.cuda(), torch.arange(n).cuda())
    table = torch.arange(cache.n_pages, dtype=torch.int32).view(1, -1).cuda()
    refs = [(kv_ref.values(*kv_ref.quantize(x.numpy(), "Q8_0")), kv_ref.values(*kv_ref.quantize(y.numpy(), "Q8_0")))]
    out = ft.attn_kv(cache, q.cuda(), table, ints([n]), ints([0, 1]), max_kv=n)
    right(out, q, [n], [1], refs, dtype)
    short = ft.attn_kv(cache, q.cuda(), table, ints([40000]), ints([0, 1]), max_kv=n)   # the last parts hold no key
    right(short, q, [40000], [1], refs, dtype)
    assert torch.equal(out, ft.attn_kv(cache, q.cuda(), table, ints([n]), ints([0, 1]), max_kv=n))


@pytest.mark.parametrize("new,k,v", [([1, 1], "Q8_0", "Q4_0"), ([3, 1], "Q4_0", "Q8_0"), ([60, 1], "Q8_0", "Q8_0")])
def test_captured_split_steps(new, k, v):
    """Store and attend, captured once with split keys and replayed while the lengths on the device grow, over borders of
    steps and parts; two graphs with a workspace each replay on two streams at once, eager calls between."""
    page, heads, heads_kv, dim, max_kv = 16, 4, 2, 64, 3000
    kv = [250, 1400]
    cache, table, refs = build([max_kv, max_kv], heads_kv, dim, page, k, v, 32)
    n = ft.attn_kv_scratch_bytes(cache, sum(new), heads, 2, max_kv)
    assert n > 0
    t = sum(new)
    lens, slots = ints(kv), torch.zeros(t, dtype=torch.int64, device="cuda")
    x, y = (torch.zeros(t, heads_kv, dim, device="cuda") for _ in range(2))
    q, start = torch.zeros(t, heads, dim, device="cuda"), ints(np.concatenate([[0], np.cumsum(new)]))
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        ws, out, s = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ft.kv_store(cache, x, y, slots, stream=s)
            ft.attn_kv(cache, q, table, lens, start, max_kv=max_kv, out=out, workspace=ws, stream=s)
        graphs.append((graph, s, ws, out))
    tab, gen = table.cpu().numpy(), torch.Generator().manual_seed(1)
    for step in (1, 5, 700, 63, 64, 300):
        where = []
        for i in range(2):
            kv[i] += max(step, new[i])
            j = np.arange(kv[i] - new[i], kv[i])
            where.append(tab[i, j // page].astype(np.int64) * page + j % page)
        slots.copy_(torch.from_numpy(np.concatenate(where)))
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        for z in (x, y, q):
            z.copy_(torch.randn(z.shape, generator=gen))
        first = 0
        for i in range(2):   # what the slots stand for now
            a = slice(kv[i] - new[i], kv[i])
            for z, ty, ref in ((x, k, refs[i][0]), (y, v, refs[i][1])):
                ref[a] = kv_ref.values(*kv_ref.quantize(z[first:first + new[i]].cpu().numpy(), ty))
            first += new[i]
        torch.cuda.synchronize()
        for graph, s, _, out in graphs:
            out.fill_(9.0)
        torch.cuda.synchronize()
        for graph, s, _, out in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        want = ft.attn_kv(cache, q, table, lens, start, max_kv=max_kv)
        for graph, s, _, out in graphs:
            assert torch.equal(out, want), step
        right(want, q, kv, new, refs, "f32")
