"""GPU: keys that no row sees leave no trace in the attention, whatever their slots hold: pages that a window has left
behind, the columns below a shared prefix in the other sequences' table rows.  Such columns hold -1 here (clamped to
page 0), and page 0 holds scales that are NaN or as large as fp16 goes, next to scales of about 2^-6."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import kv_ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FILLS = {"nan": 0xFF, "large": 0x7B}   # fp16 NaN, and 0x7B7B = 61280


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def check(kv, new, heads, heads_kv, dim, fill, dtype, page=16, k="Q8_0", v="Q8_0", window=0, prefix=0, shared=0, causal=True, seed=0):
    """Every page that some row sees is written; table columns of all others are -1."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    held = shared // page
    need = [max(0, -(-n // page) - held) for n in kv]
    n_pages = 1 + held + sum(need)
    order = 1 + rng.permutation(n_pages - 1)
    table = np.full((len(kv), max(-(-n // page) for n in kv)), -1, np.int32)
    table[0, :held] = order[:held]
    at = held
    cache = ft.KvCache.empty(n_pages, page, heads_kv, dim, k, v)
    for pool in (cache.k_pages, cache.v_pages):
        pool.fill_(FILLS[fill])
    common = torch.randn(2, shared, heads_kv, dim, generator=g)
    refs, first = [], []
    for i, (n, c, pages) in enumerate(zip(kv, new, need)):
        table[i, held:held + pages] = order[at:at + pages]
        at += pages
        x, y = torch.randn(2, n, heads_kv, dim, generator=g)
        x[:shared], y[:shared] = common
        j = np.arange(n)
        whose = np.where(j < shared, table[0, j // page], table[i, j // page])
        ft.kv_store(cache, x.cuda(), y.cuda(), torch.from_numpy(whose.astype(np.int64) * page + j % page).cuda())
        refs.append((kv_ref.values(*kv_ref.quantize(x.numpy(), k)), kv_ref.values(*kv_ref.quantize(y.numpy(), v))))
        oldest = max(0, n - c - window + 1) if window else 0   # the first key that any row's window holds
        first.append(oldest)
        for col in range(-(-prefix // page), oldest // page):
            # the page is free again: what it held is gone
            if table[i, col] > 0:
                cache.k_pages[table[i, col]].fill_(FILLS[fill])
                cache.v_pages[table[i, col]].fill_(FILLS[fill])
            table[i, col] = -1
    q = torch.randn(sum(new), heads, dim, generator=g).to(TYPES[dtype])
    start = np.concatenate([[0], np.cumsum(new)])
    ints = dict(dtype=torch.int32, device="cuda")
    out = ft.attn_kv(cache, q.cuda(), torch.from_numpy(table).cuda(), torch.tensor(kv, **ints), torch.tensor(start, **ints), window=window,
                     causal=causal, n_shared=shared, prefix_len=torch.full((len(kv),), prefix, **ints) if prefix else None)
    got = out.double().cpu().numpy()
    for i, (n, c) in enumerate(zip(kv, new)):
        a = slice(start[i], start[i + 1])
        o, terms, bias, mass = kv_ref.attention(q[a].double().numpy(), *refs[i], c, n, window=window, prefix=min(prefix, n), causal=causal)
        seen = np.concatenate([refs[i][1][:prefix], refs[i][1][max(prefix, first[i]):]])   # of what the bound's largest value is
        bound = kv_ref.attention_bound(o, terms, bias, mass, seen, dtype)
        off = np.abs(got[a] - o)
        assert np.all(np.isfinite(got[a])), f"sequence {i}: {np.sum(~np.isfinite(got[a]))} outputs are not finite"
        assert np.all(off <= bound), f"sequence {i}: {np.sum(off > bound)} outputs off, by up to {np.max(off / bound)} bounds"


@pytest.mark.parametrize("fill", list(FILLS))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kv,new,kw", [([300, 140], [1, 1], dict(window=70)), ([300, 171], [2, 3], dict(window=37, prefix=20)),
                                       ([1500], [1], dict(window=1201)), ([190, 77], [130, 40], dict(window=25)),
                                       ([400, 390], [140, 120], dict(window=90, prefix=4)), ([2000], [300], dict(window=530))])
def test_behind_a_window(kv, new, kw, dtype, fill):
    check(kv, new, 4, 2, 64, fill, dtype, **kw)
    check(kv, new, 4, 2, 128, fill, dtype, k="Q4_0", v="Q4_0", causal=False, **kw)


@pytest.mark.parametrize("fill", list(FILLS))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shared", [16, 80])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 3, 2], [20, 40, 1], [150, 140, 130]])
def test_below_a_shared_prefix(new, shared, dtype, fill):
    kv = [shared + 190, shared + 150, shared + 130]
    check(kv, new, 6, 2, 64, fill, dtype, shared=shared)
    check(kv, new, 6, 2, 96, fill, dtype, shared=shared, v="Q4_0")


@pytest.mark.parametrize("fill", list(FILLS))
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_tall_tiles(dim, dtype, fill):
    """Rows enough for the kernel with two row operands per wave (bf16 at head size 128)."""
    check([500], [264], 128, 4, dim, fill, dtype, window=40)
