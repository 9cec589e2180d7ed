"""GPU: attention over the paged cache against its plain 64-bit form (bounds: kv_ref.attention_bound)."""
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


def build(kv, heads_kv, dim, page, k, v, seed, shared=0, size=1.0, extra=2):
    """A cache with every sequence's keys stored through ft.kv_store, its table, and the values it stands for (per
    sequence, float64).  Slots that no key was written to hold 0xFF bytes: NaN scales."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    held = shared // page
    need = [max(0, -(-n // page) - held) for n in kv]
    n_pages = held + sum(need) + extra
    order = rng.permutation(n_pages)
    cols = max(1, max(-(-n // page) for n in kv), held)
    table = np.full((len(kv), cols), 10 ** 6, np.int32)       # columns past a sequence's pages: not ids
    at = held
    for i, c in enumerate(need):
        table[i, :held] = order[:held]
        table[i, held:held + c] = order[at:at + c]
        at += c
    if held:
        table[0, :held] = order[:held]
    cache = ft.KvCache.empty(n_pages, page, heads_kv, dim, k, v)
    cache.k_pages.fill_(0xFF)
    cache.v_pages.fill_(0xFF)
    refs = []
    base = None
    for i, n in enumerate(kv):
        x = torch.randn(n, heads_kv, dim, generator=g) * size
        y = torch.randn(n, heads_kv, dim, generator=g) * torch.exp(torch.randn(n, heads_kv, 1, generator=g))
        if shared:
            if base is None:
                base = (torch.randn(shared, heads_kv, dim, generator=g) * size, torch.randn(shared, heads_kv, dim, generator=g))
            m = min(n, shared)
            x[:m], y[:m] = base[0][:m], base[1][:m]
        if n:
            j = np.arange(n)
            slots = table[i, j // page].astype(np.int64) * page + j % page
            ft.kv_store(cache, x.cuda(), y.cuda(), torch.from_numpy(slots).cuda())
        refs.append((kv_ref.values(*kv_ref.quantize(x.numpy(), k)), kv_ref.values(*kv_ref.quantize(y.numpy(), v))))
    return cache, torch.from_numpy(table).cuda(), refs


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(kv, new, heads, heads_kv, dim, page=16, k="Q8_0", v="Q8_0", dtype="f32", seed=0, shared=0, slopes=None, prefix=None, size=1.0,
          max_kv=None, q_of=None, **kw):
    cache, table, refs = build(kv, heads_kv, dim, page, k, v, seed, shared, size)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(sum(new), heads, dim, generator=g).to(TYPES[dtype])
    dq = q.cuda() if q_of is None else q_of(q.cuda())
    start = np.concatenate([[0], np.cumsum(new)])
    out = ft.attn_kv(cache, dq, table, ints(kv), ints(start), max_kv=max_kv, n_shared=shared,
                     slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda(),
                     prefix_len=None if prefix is None else ints(prefix), **kw)
    got = out.float().cpu().numpy().astype(np.float64)
    ref_kw = {a: b for a, b in kw.items() if a in ("scale", "causal", "window", "softcap")}
    sl = None if slopes is None else np.asarray(slopes, np.float32).astype(np.float64)
    x = q.double().numpy()
    for i, (n, c) in enumerate(zip(kv, new)):
        a = slice(start[i], start[i + 1])
        o, terms, bias, mass = kv_ref.attention(x[a], *refs[i], c, n, slopes=sl, prefix=0 if prefix is None else min(prefix[i], n), **ref_kw)
        bound = kv_ref.attention_bound(o, terms, bias, mass, refs[i][1], dtype, kw.get("softcap", 0.0))
        off = np.abs(got[a] - o)
        fine = bool(np.all(np.isfinite(got[a])) and np.all(off <= bound))
        worst = np.unravel_index(np.argmax(np.nan_to_num(off / bound, nan=np.inf)), off.shape)
        assert fine, f"sequence {i} (kv {n}, new {c}): {np.sum(~(off <= bound))} outputs, the worst at {worst}: {got[a][worst]} for {o[worst]}, bound {bound[worst]}"
    return out


PAIRS = [("Q8_0", "Q8_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0"), ("Q4_0", "Q4_0")]


@pytest.mark.parametrize("k,v", PAIRS)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_one_token(k, v, dim, dtype):
    check([1, 77, 130], [1, 1, 1], 6, 2, dim, k=k, v=v, dtype=dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 255, 257, 700])
def test_lengths_and_pages(page, n):
    check([n], [1], 4, 1, 64, page=page, k="Q4_0")


@pytest.mark.parametrize("heads,heads_kv", [(1, 1), (3, 3), (8, 1), (7, 1), (17, 1), (40, 2), (32, 8)])
def test_head_groups(heads, heads_kv):
    check([90, 300], [1, 3], heads, heads_kv, 64)


@pytest.mark.parametrize("k,v", PAIRS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kv,new", [([33], [33]), ([200], [130]), ([5, 130, 64, 1], [5, 70, 1, 1])])
def test_prompts(kv, new, k, v, dtype):
    check(kv, new, 4, 2, 128, page=32, k=k, v=v, dtype=dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kv,new,heads,heads_kv,kw", [
    ([700], [600], 4, 1, dict()), ([257], [257], 8, 1, dict(page=64, k="Q4_0")), ([600, 9, 400, 30], [300, 9, 200, 1], 6, 2, dict(v="Q4_0")),
    ([1500], [100], 4, 1, dict(page=128)), ([500, 300], [260, 300], 2, 1, dict(window=70)), ([400], [200], 4, 1, dict(window=33, prefix=[5])),
    ([300, 280], [299, 130], 2, 2, dict(causal=False)), ([350], [350], 2, 1, dict(prefix=[200], softcap=3.0, slopes=[0.25, 0.01])),
    ([90, 64], [90, 64], 40, 1, dict(scale=-0.2)), ([30, 250], [60, 250], 2, 1, dict())])
def test_many_rows(kv, new, heads, heads_kv, kw, dtype):
    """Tiles of many rows, next to sequences of few; more new tokens than keys in the last."""
    check(kv, new, heads, heads_kv, 128, dtype=dtype, **kw)


@pytest.mark.parametrize("k,v", PAIRS)
@pytest.mark.parametrize("dim", [64, 96, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_many_rows_dims(k, v, dim, dtype):
    check([330], [290], 3, 1, dim, k=k, v=v, dtype=dtype)


def test_prompts_and_steps_together():
    """One prompt among single tokens with long contexts (their keys are split)."""
    check([900, 2500, 800, 1300], [700, 1, 1, 2], 4, 2, 64, page=32)
    check([2600, 2500, 10], [90, 1, 1], 4, 2, 64, page=32, dtype="bf16")


@pytest.mark.parametrize("dim", [64, 96, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_prompt_dims(dim, dtype):
    check([150, 70], [110, 70], 6, 2, dim, page=16, k="Q8_0", v="Q4_0", dtype=dtype)


@pytest.mark.parametrize("new", [[1, 1], [50, 9], [140, 140]])
@pytest.mark.parametrize("window", [1, 5, 64, 100, 10 ** 12])
@pytest.mark.parametrize("prefix", [None, [0, 4], [70, 200]])
def test_windows_and_prefixes(new, window, prefix):
    check([300, 140], new, 4, 2, 64, window=window, prefix=prefix)


@pytest.mark.parametrize("new", [[1, 2, 6], [60, 17, 33]])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_bidirectional_cap_and_bias(new, dtype):
    kv, sl = [100, 64, 33], [0.5, 0.25, 2.0 ** -8, 0.0]
    check(kv, new, 4, 2, 64, causal=False, dtype=dtype)
    check(kv, new, 4, 2, 64, causal=False, window=20, dtype=dtype)
    check(kv, new, 4, 2, 64, softcap=2.0, dtype=dtype)
    check(kv, new, 4, 2, 64, slopes=sl, dtype=dtype)
    check(kv, new, 4, 2, 128, slopes=sl, softcap=30.0, window=40, prefix=[3, 3, 3], dtype=dtype, scale=0.3)
    check(kv, new, 4, 2, 64, prefix=[90, 64, 2], dtype=dtype)      # a prompt seen from both sides


def test_rows_that_see_nothing():
    """Idle slots, more new tokens than keys: zeros; tokens of no sequence stay as they were."""
    cache, table, refs = build([0, 3, 40], 2, 64, 16, "Q8_0", "Q8_0", 3)
    q = torch.randn(12, 4, 64, device="cuda")
    out = torch.full_like(q, 9.0)
    ft.attn_kv(cache, q, table, ints([0, 3, 40]), ints([1, 3, 8, 10]), out=out)
    got = host(out)
    assert (got[0] == 9).all() and (got[10:] == 9).all()
    assert (got[1:3] == 0).all()                      # no keys at all
    assert (got[3:5] == 0).all() and (got[5:8] != 0).any()   # five tokens, three keys: the first two see none
    o, terms, bias, mass = kv_ref.attention(host(q)[5:8].astype(np.float64), *refs[1], 3, 3)
    assert np.all(np.abs(got[5:8] - o) <= kv_ref.attention_bound(o, terms, bias, mass, refs[1][1], "f32"))


def test_long_cache_splits():
    out = check([3000, 2111, 64, 0], [1, 2, 1, 1], 8, 2, 128, page=64, k="Q8_0", v="Q4_0")
    again = check([3000, 2111, 64, 0], [1, 2, 1, 1], 8, 2, 128, page=64, k="Q8_0", v="Q4_0")
    assert torch.equal(out, again)                    # the same bits every time


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kv,new,page,shared", [([70, 65, 200], [1, 1, 1], 16, 64), ([200, 300, 150, 129], [3, 1, 20, 1], 32, 96),
                                                ([1100, 1025], [1, 4], 128, 1024), ([64, 64], [1, 1], 64, 64), ([40, 150, 10], [1, 1, 3], 32, 96)])
def test_shared_prefix(kv, new, page, shared, dtype):
    """The last: sequences shorter than the prefix that the others share."""
    check(kv, new, 8, 2, 64, page=page, shared=shared, dtype=dtype)
    check([n + 130 for n in kv], [c + 120 for c in new], 4, 2, 64, page=page, shared=shared, dtype=dtype)   # prompts behind a shared prefix
    check(kv, new, 6, 1, 128, page=page, shared=shared, dtype=dtype, k="Q4_0", v="Q4_0", softcap=20.0, window=90, prefix=[4] * len(kv))


def test_many_sequences():
    n = 150
    rng = np.random.default_rng(0)
    kv = rng.integers(1, 90, n).tolist()
    check(kv, [min(int(a), int(b)) for a, b in zip(rng.integers(1, 4, n), kv)], 4, 2, 64, dtype="f16")


def test_uneven_scales():
    """Large and tiny scores, and V blocks whose scales lie far apart, stay within the bound."""
    heads_kv, dim, page, n = 1, 64, 16, 200
    g = torch.Generator().manual_seed(9)
    for size in (1e-20, 1e-6, 6.0, 2000.0):
        cache = ft.KvCache.empty(n // page + 1, page, heads_kv, dim)
        x = torch.randn(n, 1, dim, generator=g)
        y = torch.randn(n, 1, dim, generator=g) * torch.pow(10.0, torch.randint(-4, 5, (n, 1, 1), generator=g).float())
        ft.kv_store(cache, x.cuda(), y.cuda(), torch.arange(n).cuda())
        q = torch.randn(1, 4, dim, generator=g) * size
        table = torch.arange(n // page + 1, dtype=torch.int32).view(1, -1).cuda()
        got = host(ft.attn_kv(cache, q.cuda(), table, ints([n]), ints([0, 1]))).astype(np.float64)
        kk, vv = kv_ref.values(*kv_ref.quantize(x.numpy(), "Q8_0")), kv_ref.values(*kv_ref.quantize(y.numpy(), "Q8_0"))
        o, terms, bias, mass = kv_ref.attention(q.double().numpy(), kk, vv, 1, n)
        bound = kv_ref.attention_bound(o, terms, bias, mass, vv, "f32")
        assert np.all(np.isfinite(got)) and np.all(np.abs(got - o) <= bound), size


@pytest.mark.parametrize("dtype", list(TYPES))
def test_strided_q_and_out(dtype):
    def wide(q):   # columns of a wider row, not 16-byte aligned
        n, h, d = q.shape
        buf = torch.zeros(n, 3 + h * d, dtype=q.dtype, device=q.device)
        buf[:, 3:] = q.flatten(1)
        return buf[:, 3:].unflatten(1, (h, d))

    a = check([100, 80], [1, 40], 4, 2, 64, dtype=dtype, q_of=wide)
    b = check([100, 80], [1, 40], 4, 2, 64, dtype=dtype, q_of=lambda q: q.transpose(0, 1).contiguous().transpose(0, 1),
              out=torch.empty(4, 41, 66, dtype=TYPES[dtype], device="cuda")[:, :, 1:65].transpose(0, 1))
    assert torch.equal(a, b)


def test_bounds_of_the_host():
    """Lengths past max_kv or past the table are cut to it; an id outside the pool is clamped."""
    cache, table, refs = build([100], 1, 64, 16, "Q8_0", "Q8_0", 5)
    q = torch.randn(1, 2, 64, device="cuda")
    cut = ft.attn_kv(cache, q, table, ints([100]), ints([0, 1]), max_kv=64)
    want = ft.attn_kv(cache, q, table, ints([64]), ints([0, 1]))
    assert torch.equal(cut, want)
    long = ft.attn_kv(cache, q, table, ints([10 ** 6]), ints([0, 1]), max_kv=10 ** 6)
    assert long.shape == q.shape
    bad = table.clone()
    bad[0, 0], bad[0, 1] = -5, 2 ** 30
    ft.attn_kv(cache, q, bad, ints([100]), ints([0, 1]))
    ft.attn_kv(cache, q, table, ints([-7]), ints([0, 1]))
    ft.attn_kv(cache, q, table, ints([50]), ints([-3, 1000]))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("new,heads,max_kv,shared", [([130], 32, 6000, 0), ([300], 32, 3000, 0), ([20, 130, 1], 32, 2000, 0),
                                                     ([1] * 20, 32, 3000, 1024), ([2], 32, 9000, 0)])
def test_a_workspace_holds_every_type(new, heads, max_kv, shared, dtype):
    """The split of the keys depends on the type, the workspace's size does not."""
    kv = [shared + max(new) + 70] * len(new)
    cache, table, _ = build(kv, 8, 128, 16, "Q8_0", "Q8_0", 5, shared)
    table = torch.cat([table, torch.zeros(len(new), max_kv // 16, dtype=torch.int32, device="cuda")], 1).contiguous()
    q = torch.randn(sum(new), heads, 128, generator=torch.Generator().manual_seed(6)).to(TYPES[dtype]).cuda()
    args = (cache, q, table, ints(kv), ints(np.concatenate([[0], np.cumsum(new)])))
    want = ft.attn_kv(*args, max_kv=max_kv, n_shared=shared)
    ws = torch.empty(ft.attn_kv_scratch_bytes(cache, sum(new), heads, len(new), max_kv, n_shared=shared), dtype=torch.uint8, device="cuda")
    assert torch.equal(ft.attn_kv(*args, max_kv=max_kv, n_shared=shared, workspace=ws if ws.numel() else None), want)


# rows enough that the kernel with two row operands per wave is taken (two workgroups per CU of the other would be
# slower): 264 tokens of 32 query heads per key/value head
@pytest.mark.parametrize("k,v", PAIRS)
def test_many_rows_of_bf16(k, v):
    check([500], [264], 128, 4, 128, k=k, v=v, dtype="bf16", causal=False)


@pytest.mark.parametrize("kv,new,kw", [([2900], [264], dict(softcap=20.0, max_kv=3000)),
                                       ([590, 450, 3], [150, 130, 3], dict(causal=False, slopes=[0.5 / (1 + h) for h in range(128)])),
                                       ([700], [270], dict(causal=False, window=300, prefix=[40]))])
def test_masks_of_many_rows_of_bf16(kv, new, kw):
    check(kv, new, 128, 4, 128, dtype="bf16", **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_cap_far_below_every_score(dtype):
    """cap * tanh(s / cap) with a cap of 1e-37 and q rows of large and zero elements: all visible keys weigh alike."""
    cache, table, refs = build([70], 1, 64, 16, "Q8_0", "Q8_0", 9)
    q = torch.zeros(2, 2, 64)
    q[0] = 1e4
    out = ft.attn_kv(cache, q.to(TYPES[dtype]).cuda(), table, ints([70]), ints([0, 2]), causal=False, softcap=1e-37, scale=1e3)
    mean = refs[0][1].mean(0)[0]
    # the weights' sum in 32 bits (70 terms), their product with V's scales and the output's rounding at half a step each
    tol = {"f32": 2 ** -17, "f16": 2 ** -10, "bf16": 2 ** -7}[dtype] * np.abs(refs[0][1]).mean(0)[0]
    assert np.all(np.abs(out.double().cpu().numpy() - mean) <= tol)


def test_workspace_and_streams():
    kv = [2000, 900]
    cache, table, _ = build(kv, 2, 64, 32, "Q8_0", "Q8_0", 6)
    q = torch.randn(2, 4, 64, device="cuda")
    args = (cache, q, table, ints(kv), ints([0, 1, 2]))
    want = ft.attn_kv(*args, max_kv=2000)
    n = ft.attn_kv_scratch_bytes(cache, 2, 4, 2, 2000)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(ft.attn_kv(*args, max_kv=2000, workspace=ws), want)
    with pytest.raises(ft.FtError):
        ft.attn_kv(*args, max_kv=2000, workspace=ws[:n // 2])
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [ft.attn_kv(*args, max_kv=2000, stream=x) for _ in range(4) for x in s]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_captured_step():
    """A decode step (store, attend) captured once and replayed while the lengths on the device grow; two graphs with a
    workspace each replay on two streams at once."""
    kv, page, heads, heads_kv, dim = [130, 40], 16, 4, 2, 64
    cache, table, _ = build([190, 190], heads_kv, dim, page, "Q8_0", "Q4_0", 7)
    max_kv = 190
    n = ft.attn_kv_scratch_bytes(cache, 2, heads, 2, max_kv)
    lens, slots = ints(kv), torch.zeros(2, dtype=torch.int64, device="cuda")
    k, v = (torch.zeros(2, heads_kv, dim, device="cuda") for _ in range(2))
    q = torch.zeros(2, heads, dim, device="cuda")
    start = ints([0, 1, 2])
    graphs, outs = [], []
    for _ in range(2):
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            ft.kv_store(cache, k, v, slots, stream=s)
            ft.attn_kv(cache, q, table, lens, start, max_kv=max_kv, out=out, workspace=ws, stream=s)
        graphs.append((gr, s, ws))
        outs.append(out)
    tab = table.cpu().numpy()
    gen = torch.Generator().manual_seed(1)
    for step in range(4):
        for i in range(2):
            kv[i] += 1
            j = kv[i] - 1
            slots[i] = int(tab[i, j // page]) * page + j % page
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=gen))
        torch.cuda.synchronize()
        for gr, s, _ in graphs:
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        ft.kv_store(cache, k, v, slots)
        want = ft.attn_kv(cache, q, table, lens, start, max_kv=max_kv)
        for out in outs:
            assert torch.equal(out, want), step


def test_refusals_of_the_binding():
    cache, table, _ = build([20], 2, 64, 16, "Q8_0", "Q8_0", 8)
    q = torch.randn(1, 4, 64, device="cuda")
    ok = (cache, q, table, ints([20]), ints([0, 1]))
    ft.attn_kv(*ok)
    for i, bad in ((1, q[..., :32]), (1, q.double()), (1, q.cpu()), (2, table.long()), (2, table.cpu()), (3, ints([20, 1])),
                   (4, ints([0])), (4, ints([0, 1]).long())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            ft.attn_kv(*args)
    for kw in (dict(slopes=torch.ones(3, device="cuda")), dict(prefix_len=ints([1, 2])), dict(out=q.half()), dict(scale=0.0)):
        with pytest.raises(ValueError):
            ft.attn_kv(*ok, **kw)
    with pytest.raises(ft.FtError):
        ft.attn_kv(*ok, n_shared=8)
    with pytest.raises(ValueError):
        ft.KvCache(cache.k_pages[:, :-1].contiguous(), cache.v_pages, 16, 2, 64)
    with pytest.raises(ValueError):
        ft.kv_store(cache, q, q, torch.zeros(1, dtype=torch.int64, device="cuda"))
