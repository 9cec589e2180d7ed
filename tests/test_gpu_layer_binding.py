"""GPU: what ft.rope, ft.kv_store_rope, ft.kv_load, ft.norm and ft.lora refuse of their tensors before the library is
called, and the objects that they return."""
import gc
import weakref

import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

T, H, D, W = 3, 4, 64, 96


def some(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype, device="cuda")


def rope():
    return ft.rope, dict(x=some(T, H, D), positions=some(T, dtype=torch.int32), table=some(10, 32), weight=some(D), out=some(T, H, D))


def store():
    cache = ft.KvCache.empty(2, 16, 2, D)
    return lambda **kw: ft.kv_store_rope(cache, **kw), dict(
        q=some(T, H, D), k=some(T, 2, D), v=some(T, 2, D), slots=torch.arange(T, device="cuda"), positions=some(T, dtype=torch.int32),
        table=some(10, 32), q_weight=some(D), k_weight=some(D), q_out=some(T, H, D))


def load():
    cache = ft.KvCache.empty(2, 16, 2, D)
    ft.kv_store(cache, 127 * some(T, 2, D), 127 * some(T, 2, D), torch.arange(T, device="cuda"))
    return lambda **kw: ft.kv_load(cache, **kw), dict(slots=torch.arange(T, device="cuda"), k=some(T, 2, D), v=some(T, 2, D))


def norm():
    return ft.norm, dict(x=some(T, W), weight=some(W), bias=some(W), residual=some(T, W), post_weight=some(W), post_bias=some(W), gate=some(T, W),
                         act="Q8_1", r=some(T, W), out=some(T, W), xq=some(T, W // 32 * 36, dtype=torch.uint8))


def lora():
    return ft.lora, dict(x=some(T, W), a=some(5, 8, W), b=some(5, 16, 8), ids=some(T, dtype=torch.int32), y=some(T, 16), scales=some(5),
                         ranks=some(5, dtype=torch.int32), out=some(T, 16),
                         workspace=some(ft.lora_scratch_bytes(T, W, 5, 8), dtype=torch.uint8))


@pytest.mark.parametrize("make", (rope, store, load, norm, lora))
def test_wrong_tensors_refused(make):
    need_gpu()
    f, good = make()
    f(**good)
    for name, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = {"host": t.cpu(), "number": 1.0, "elements apart": torch.stack([t, t], -1)[..., 0]}
        if name == "workspace":
            bad["short"] = t[:16]
        else:
            bad.update(type=t.to(torch.float64), one_more=torch.cat([t, t[:1]]), axis=t.unsqueeze(0))
            if name == "table":
                del bad["one_more"]    # a longer table is a table
            if name in ("a", "b"):
                bad["wide"] = torch.cat([t, t], -1)
        for why, wrong in bad.items():
            with pytest.raises((ValueError, TypeError, ft.FtError)):
                f(**{**good, name: wrong})
                pytest.fail(f"{name}: {why}")
    torch.cuda.synchronize()
    f(**good)


def test_refusals_name_their_cause():
    need_gpu()
    x, at, table = some(T, H, D), some(T, dtype=torch.int32), some(10, 32)
    with pytest.raises(ValueError, match="positions must be a contiguous"):
        ft.rope(x, at[:2], table)
    with pytest.raises(ValueError, match="out must be"):
        ft.rope(x, at, table, out=some(T, H, D, dtype=torch.float16))
    with pytest.raises(TypeError, match="table must be a tensor"):
        ft.rope(x, at, None)
    with pytest.raises(ft.FtError, match="ft_rope: FT_ERR_SHAPE") as e:
        ft.rope(x, at, some(10, 128))
    assert ft.STATUS[e.value.status] == "FT_ERR_SHAPE"
    with pytest.raises(ValueError, match="scale must not be 0"):
        ft.norm(some(T, W), scale=0.0)
    with pytest.raises(ValueError, match="xq needs an act"):
        ft.norm(some(T, W), xq=some(T, 108, dtype=torch.uint8))
    with pytest.raises(ValueError, match="q_out and q_weight are q's"):
        ft.kv_store_rope(ft.KvCache.empty(2, 16, 2, D), None, x[:, :2], x[:, :2], torch.arange(T, device="cuda"), at, table, q_weight=some(D))
    with pytest.raises((TypeError, AttributeError)):
        ft.rope(x, at, table, stream=3)


@pytest.mark.parametrize("make", (rope, store, load, norm, lora))
def test_given_tensors_come_back(make):
    """What was given is returned itself and kept by nobody; what was not is new, of its own, and needs no gradient."""
    need_gpu()
    f, good = make()
    outs = [n for n in (("k", "v") if make is load else ("r", "q_out", "out", "xq")) if n in good]
    got = f(**good)
    got = got if isinstance(got, tuple) else (got,)
    assert all(a is good[n] for a, n in zip(got, outs)) and len(got) == len(outs)
    refs = [weakref.ref(good[n]) for n in outs]
    rest = {n: t.requires_grad_() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for n, t in good.items() if n not in outs}
    del good, got
    gc.collect()
    assert all(r() is None for r in refs)
    if f is ft.norm:
        rest["rows"] = True
    new = f(**rest)
    new = new if isinstance(new, tuple) else (new,)
    assert len(new) == len(outs) and not any(t.requires_grad for t in new)
    assert all(t.is_contiguous() for t in new)
    again = f(**rest)
    again = again if isinstance(again, tuple) else (again,)
    torch.cuda.synchronize()
    for a, b in zip(new, again):
        assert a.data_ptr() != b.data_ptr() and torch.equal(a, b)


def test_what_norm_returns():
    need_gpu()
    x, w = some(T, W), some(W)
    r, n, xq = ft.norm(x, w)
    assert r is x and n.shape == x.shape and xq is None
    r, n, xq = ft.norm(x, w, act="Q8_0")
    assert r is x and n is None and xq.shape == (T, W // 32 * 34) and xq.dtype is torch.uint8
    r, n, xq = ft.norm(x, w, residual=x, act="Q8_0", rows=True)
    assert r is not x and n is not None and xq is not None and torch.equal(r, 2 * x)
    for gate in (2 * some(W), 2 * some(1, W), (2 * some(1, W)).expand(T, W), 2 * some(T, W)):
        assert torch.equal(ft.norm(x, w, gate=gate)[0], 2 * x)
    with pytest.raises(ValueError):
        ft.norm(x, w, gate=some(2, W))


def test_without_queries():
    need_gpu()
    x = some(T, 2, D)
    cache = ft.KvCache.empty(2, 16, 2, D)
    assert ft.kv_store_rope(cache, None, x, x, torch.arange(T, device="cuda"), some(T, dtype=torch.int32), some(10, 32)) is None


def test_what_a_load_returns():
    need_gpu()
    f, good = load()
    for kw, dtype in ((dict(), torch.float32), (dict(dtype=torch.float16), torch.float16), (dict(v=some(T, 2, D, dtype=torch.bfloat16)), torch.bfloat16)):
        k, v = f(slots=good["slots"], **kw)
        assert k.dtype is v.dtype is dtype and k.shape == v.shape == (T, 2, D) and torch.equal(k, torch.full_like(k, 127)) and torch.equal(v, k)
    for kw in (dict(dtype=torch.float64), dict(k=good["k"], v=some(T, 2, D, dtype=torch.float16)), dict(dtype="float32")):
        with pytest.raises((ValueError, TypeError)):
            f(slots=good["slots"], **kw)


def test_no_tokens():
    need_gpu()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ft.rope(some(0, H, D), none, some(10, 32)).shape == (0, H, D)
    assert [None if t is None else tuple(t.shape) for t in ft.norm(some(0, W), act="Q8_1")] == [(0, W), None, (0, W // 32 * 36)]
    assert ft.lora(some(0, W), some(5, 8, W), some(5, 16, 8), none).shape == (0, 16)
    q = ft.kv_store_rope(ft.KvCache.empty(2, 16, 2, D), some(0, H, D), some(0, 2, D), some(0, 2, D), none.long(), none, some(10, 32))
    assert q.shape == (0, H, D)
