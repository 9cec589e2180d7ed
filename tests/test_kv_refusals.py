"""Host-side refusals of the key/value cache, its attention and the scored router (no
GPU: every call is refused before anything is enqueued)."""
import ctypes

import pytest
import torch

from block_quantized_matvec_amd import ft

ST = {v: k for k, v in ft.STATUS.items()}
FAKE, ODD = 1 << 20, (1 << 20) + 2


def cache(**kw):
    f = dict(k_type=1, v_type=0, k_pages=FAKE, v_pages=FAKE, n_pages=4, page_size=16, n_kv_head=2, head_dim=64)
    f.update(kw)
    return ft._KvCache(*f.values())


def status(name, *args):
    return ft.STATUS[getattr(ft.lib(), name)(*args)]


def store(c=None, ty=0, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, slots=FAKE, t=2):
    return status("ft_kv_store", ctypes.byref(c or cache()), ty, k, kt, kh, v, vt, vh, slots, t, None)


def load(c=None, ty=0, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, slots=FAKE, t=2):
    return status("ft_kv_load", ctypes.byref(c or cache()), slots, t, ty, k, kt, kh, v, vt, vh, None)


def attn(c=None, ty=0, q=FAKE, qt=256, qh=64, n_tok=2, n_head=4, q_start=FAKE, kv_len=FAKE, table=FAKE, ld=4, cols=4,
         n_seq=2, max_kv=64, out=FAKE, ot=256, oh=64, **o):
    f = dict(scale=0.0, softcap=0.0, bidirectional=0, window=0, slopes=None, prefix_len=None, n_shared=0, workspace=None,
             workspace_bytes=0)
    f.update(o)
    return status("ft_attn_kv", ctypes.byref(c or cache()), ty, q, qt, qh, n_tok, n_head, q_start, kv_len, table, ld, cols,
                  n_seq, max_kv, out, ot, oh, ctypes.byref(ft._AttnOpts(*f.values())), None)


def route(x=FAKE, ty=0, t=2, e=64, ld=64, topk=4, ids=FAKE, w=FAKE, **o):
    f = dict(sigmoid=0, bias=None, n_group=0, topk_group=0, group_top=0, no_renorm=0, scale=0.0)
    f.update(o)
    return status("ft_moe_route_ex", x, ty, t, e, ld, topk, ctypes.byref(ft._RouteOpts(*f.values())), ids, w, None)


@pytest.mark.parametrize("call", [store, load, attn])
def test_cache_refused(call):
    assert call(cache(k_type=2)) == "FT_ERR_UNSUPPORTED"
    assert call(cache(v_type=6)) == "FT_ERR_UNSUPPORTED"
    for bad in (dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(head_dim=80), dict(head_dim=0),
                dict(n_kv_head=0), dict(n_kv_head=1025), dict(n_pages=0), dict(n_pages=1 << 31)):
        assert call(cache(**bad)) == "FT_ERR_SHAPE", bad
    assert call(cache(k_pages=None)) == "FT_ERR_INVALID_ARG"
    assert call(cache(v_pages=FAKE + 8)) == "FT_ERR_ALIGNMENT"
    assert call(ty=3) == "FT_ERR_UNSUPPORTED"


def test_page_bytes():
    for dim in (64, 96, 128, 256):
        for page in (16, 32, 64, 128, 256):
            assert ft.kv_page_bytes("Q8_0", page, 3, dim) == page * 3 * dim // 32 * 34
            assert ft.kv_page_bytes("Q4_0", page, 3, dim) == page * 3 * dim // 32 * 18
    for ty, page, heads, dim in (("Q4_K", 16, 1, 64), ("Q8_0", 24, 1, 64), ("Q8_0", 16, 0, 64), ("Q8_0", 16, 1, 32)):
        assert ft.lib().ft_kv_page_bytes(ft.TYPES[ty], page, heads, dim) == 0
        with pytest.raises(ft.FtError):
            ft.kv_page_bytes(ty, page, heads, dim)
    for k in ft.TYPES:
        for v in ft.TYPES:
            assert ft.supported("kv_cache", k, v) == (k in ("Q8_0", "Q4_0") and v in ("Q8_0", "Q4_0"))


@pytest.mark.parametrize("call", [store, load])
def test_rows_refused(call):
    assert call(t=-1) == "FT_ERR_INVALID_ARG"
    assert call(kt=63) == "FT_ERR_INVALID_ARG"
    assert call(vh=63) == "FT_ERR_INVALID_ARG"
    assert call(kh=-64) == "FT_ERR_INVALID_ARG"
    assert call(t=(1 << 24) + 1) == "FT_ERR_SHAPE"
    assert call(slots=None) == "FT_ERR_INVALID_ARG"
    assert call(slots=FAKE + 4) == "FT_ERR_ALIGNMENT"
    assert call(k=ODD) == "FT_ERR_ALIGNMENT"
    assert call(ty=1, v=ODD + 1) == "FT_ERR_ALIGNMENT"
    assert call(t=0, k=None, v=None, slots=None) == "FT_OK"


def test_store_and_load_sides():
    assert store(k=None) == "FT_ERR_INVALID_ARG"
    assert store(v=None) == "FT_ERR_INVALID_ARG"
    assert load(k=None, v=None) == "FT_OK"                       # nothing to read
    assert load(k=None, kt=0, kh=0, slots=None) == "FT_ERR_INVALID_ARG"


def test_attention_refused():
    assert attn(n_head=3) == "FT_ERR_SHAPE"
    assert attn(n_head=0) == "FT_ERR_SHAPE"
    assert attn(n_head=1026) == "FT_ERR_SHAPE"
    assert attn(qt=63) == "FT_ERR_INVALID_ARG"
    assert attn(oh=32) == "FT_ERR_INVALID_ARG"
    assert attn(cols=0) == "FT_ERR_INVALID_ARG"
    assert attn(ld=3) == "FT_ERR_INVALID_ARG"
    assert attn(max_kv=-1) == "FT_ERR_INVALID_ARG"
    assert attn(n_tok=-1) == "FT_ERR_INVALID_ARG"
    assert attn(n_tok=(1 << 24) + 1) == "FT_ERR_SHAPE"
    wide = dict(c=cache(n_kv_head=64), n_tok=1 << 24, n_head=64, qt=64 * 64, ot=64 * 64)
    assert attn(**wide) == "FT_ERR_SHAPE"                        # more rows than one launch takes
    assert attn(window=-1) == "FT_ERR_INVALID_ARG"
    for bad in (-1.0, float("nan"), float("inf")):
        assert attn(softcap=bad) == "FT_ERR_INVALID_ARG"
    assert attn(scale=float("nan")) == "FT_ERR_INVALID_ARG"
    assert attn(bidirectional=2) == "FT_ERR_INVALID_ARG"
    assert attn(n_shared=8) == "FT_ERR_SHAPE"                    # not whole pages
    assert attn(n_shared=80) == "FT_ERR_SHAPE"                   # past max_kv
    assert attn(n_shared=-16) == "FT_ERR_INVALID_ARG"
    for name in ("q", "out", "q_start", "kv_len", "table"):
        assert attn(**{name: None}) == "FT_ERR_INVALID_ARG", name
        assert attn(**{name: ODD}) == "FT_ERR_ALIGNMENT", name
    for name in ("slopes", "prefix_len"):
        assert attn(**{name: ODD}) == "FT_ERR_ALIGNMENT", name
    assert attn(workspace=FAKE + 8) == "FT_ERR_ALIGNMENT"
    # a long cache and few rows: the keys are split, which takes a workspace
    assert attn(workspace=FAKE, workspace_bytes=16, cols=1000, ld=1000, max_kv=16000) == "FT_ERR_NO_SCRATCH"
    assert attn(n_tok=0, q=None, out=None) == "FT_OK"
    assert attn(n_seq=0, q_start=None, table=None) == "FT_OK"


def test_attention_scratch():
    c = cache()
    n = lambda *a: ft.lib().ft_attn_kv_scratch_bytes(ctypes.byref(c), *a, None)  # noqa: E731
    assert n(1, 4, 1, 16000) > 0
    assert n(0, 4, 1, 16000) == 0 and n(1, 3, 1, 16000) == 0
    assert n(1 << 17, 4, 1, 1 << 17) == 0                        # enough rows: the keys stay whole


def test_route_refused():
    assert route(ty=3) == "FT_ERR_UNSUPPORTED"
    assert route(e=1025, ld=1025) == "FT_ERR_SHAPE"
    assert route(e=0, ld=0) == "FT_ERR_SHAPE"
    assert route(t=(1 << 25) + 1) == "FT_ERR_SHAPE"
    assert route(topk=0) == "FT_ERR_SHAPE"
    assert route(topk=33) == "FT_ERR_SHAPE"
    assert route(e=3, ld=3, topk=4) == "FT_ERR_SHAPE"
    assert route(n_group=7) == "FT_ERR_SHAPE"
    assert route(n_group=65) == "FT_ERR_SHAPE"
    assert route(n_group=8, topk_group=9) == "FT_ERR_SHAPE"
    assert route(n_group=32, topk_group=1, topk=3) == "FT_ERR_SHAPE"   # two experts left for three slots
    assert route(group_top=3) == "FT_ERR_INVALID_ARG"
    assert route(sigmoid=2) == "FT_ERR_INVALID_ARG"
    assert route(ld=63) == "FT_ERR_INVALID_ARG"
    assert route(scale=float("inf")) == "FT_ERR_INVALID_ARG"
    assert route(x=None) == "FT_ERR_INVALID_ARG"
    assert route(ids=None) == "FT_ERR_INVALID_ARG"
    assert route(x=ODD) == "FT_ERR_ALIGNMENT"
    assert route(t=0, x=None, ids=None, w=None) == "FT_OK"


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        ft.moe_route_ex(x, 4)
    with pytest.raises(ValueError):
        ft.KvCache(torch.zeros(ft.kv_page_bytes("Q8_0", 16, 1, 64), dtype=torch.uint8),
                   torch.zeros(ft.kv_page_bytes("Q8_0", 16, 1, 64), dtype=torch.uint8), 16, 1, 64)
