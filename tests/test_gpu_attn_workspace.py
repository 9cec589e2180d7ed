"""GPU: the size that ft.attn_kv_scratch_bytes gives holds for the call it was asked for, whatever the table's width, and
for every smaller bound of the lengths, as a workspace and as a reserved pool under capture."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import need_gpu
from tests.test_gpu_attn_kv import build, ints

pytestmark = pytest.mark.gpu

# new tokens per sequence, heads, key/value heads, the bound the size is for, the call's bound, columns of its table
# (pages of 16): calls that split the keys further than those of the larger bound
CASES = [([1], 32, 8, 16336, 16336, 1020), ([1], 32, 8, 16384, 16384, 1008), ([1], 32, 8, 131072, 16320, 1020), ([1] * 32, 32, 8, 2048, 2048, 96),
         ([5, 5, 5], 2, 1, 36296, 15276, 2300), ([1] * 8, 2, 1, 17544, 11957, 1100), ([130] * 3, 2, 1, 33245, 27962, 2100),
         ([40, 40], 8, 2, 32790, 32790, 1611), ([130] * 3, 16, 4, 21166, 16270, 1400)]


def setup(new, heads, heads_kv, cols):
    kv = [300 + 7 * i for i in range(len(new))]
    cache, table, refs = build(kv, heads_kv, 128, 16, "Q8_0", "Q8_0", 5)
    wide = torch.zeros(len(new), cols, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = torch.randn(sum(new), heads, 128, generator=torch.Generator().manual_seed(6))
    start = np.concatenate([[0], np.cumsum(new)])

    def right(out):
        out = out.double().cpu().numpy()
        for i, (n, c) in enumerate(zip(kv, new)):
            a = slice(start[i], start[i + 1])
            o, terms, bias, mass = kv_ref.attention(q[a].double().numpy(), *refs[i], c, n)
            assert np.all(np.abs(out[a] - o) <= kv_ref.attention_bound(o, terms, bias, mass, refs[i][1], "f32"))

    return cache, (cache, q.cuda(), wide, ints(kv), ints(start)), right


@pytest.mark.parametrize("new,heads,heads_kv,size_for,max_kv,cols", CASES)
def test_a_workspace(new, heads, heads_kv, size_for, max_kv, cols):
    need_gpu()
    cache, args, right = setup(new, heads, heads_kv, cols)
    ws = torch.empty(ft.attn_kv_scratch_bytes(cache, sum(new), heads, len(new), size_for), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    right(ft.attn_kv(*args, max_kv=max_kv, workspace=ws))
    right(ft.attn_kv(*args, max_kv=300 + 7 * len(new), workspace=ws))


@pytest.mark.parametrize("new,heads,heads_kv,size_for,max_kv,cols", CASES)
def test_a_pool_under_capture(new, heads, heads_kv, size_for, max_kv, cols):
    need_gpu()
    cache, args, right = setup(new, heads, heads_kv, cols)
    s = torch.cuda.Stream()
    ft.scratch_reserve(ft.attn_kv_scratch_bytes(cache, sum(new), heads, len(new), size_for), stream=s)
    out = torch.zeros(sum(new), heads, 128, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ft.attn_kv(*args, max_kv=max_kv, out=out, stream=s)
    for _ in range(3):
        out.fill_(9.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        right(out)
