"""Host-side refusals of the rotation, the store that turns, the norm and the adapters (no GPU: every call is refused
before anything is enqueued), their sizes, and the angles of long contexts."""
import ctypes
import math
import struct

import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.test_kv_refusals import FAKE, ODD, cache, status

BIG = 1 << 41
# ft_rotation, ft_qkv_rows, ft_norm_opts and ft_lora_opts; 0 is a NULL pointer
ROTATION, ROWS, NORM, LORA = (struct.Struct(f) for f in ("@PPqqi0P", "@PqqqPPqqPqqPPqqd", "@PqPqiPPfidPPPqPqiP", "@PPPN"))


def packed(struct, fields):
    return struct.pack(*(0 if v is None else v for v in fields.values()))


def rotation(**kw):
    f = dict(table=FAKE, positions=FAKE, n_pos=100, rot_dim=64, interleaved=0)
    f.update(kw)
    return packed(ROTATION, f)


def rope(rot=None, ty=0, x=FAKE, xt=256, xh=64, t=2, heads=4, dim=64, weight=None, eps=0.0, out=FAKE + 4096, ot=256, oh=64):
    return status("ft_rope", rot or rotation(), ty, x, xt, xh, t, heads, dim, weight, eps, out, ot, oh, None)


def store(c=None, rot=None, ty=0, slots=FAKE, t=2, **o):
    f = dict(q=FAKE, q_token=256, q_head=64, n_head=4, q_weight=None, q_out=FAKE + 4096, out_token=256, out_head=64, k=FAKE, k_token=128,
             k_head=64, k_weight=None, v=FAKE, v_token=128, v_head=64, eps=0.0)
    f.update(o)
    return status("ft_kv_store_rope", ctypes.byref(c or cache()), rot or rotation(), ty, packed(ROWS, f), slots, t,
                  None)


def norm(ty=0, x=FAKE, ldx=64, rows=2, width=64, **o):
    f = dict(residual=None, ld_residual=0, gate=None, ld_gate=0, post=0, post_weight=None, post_bias=None, scale=0.0, layer=0, eps=0.0,
             weight=None, bias=None, r=None, ld_r=0, out=FAKE, ld_out=64, act=0, xq=None)
    f.update(o)
    return status("ft_norm", ty, x, ldx, rows, width, packed(NORM, f), None)


def lora(tx=0, x=FAKE, ldx=64, t=2, k=64, tw=2, a=FAKE, b=FAKE, many=3, rank=16, n=32, ids=FAKE, y=FAKE, ldy=32, out=FAKE, ldo=32, **o):
    f = dict(ranks=None, scales=None, workspace=None, workspace_bytes=0)
    f.update(o)
    return status("ft_lora", tx, x, ldx, t, k, tw, a, b, many, rank, n, ids, y, ldy, out, ldo, packed(LORA, f), None)


def test_rope_refused():
    for call in (rope, store):
        assert call(ty=3) == "FT_ERR_UNSUPPORTED"
        for kw, want in ((dict(rot_dim=63), "FT_ERR_SHAPE"), (dict(rot_dim=0), "FT_ERR_SHAPE"), (dict(rot_dim=66), "FT_ERR_SHAPE"),
                         (dict(n_pos=0), "FT_ERR_INVALID_ARG"), (dict(table=None), "FT_ERR_INVALID_ARG"), (dict(table=ODD), "FT_ERR_ALIGNMENT"),
                         (dict(positions=None), "FT_ERR_INVALID_ARG"), (dict(positions=ODD), "FT_ERR_ALIGNMENT"),
                         (dict(n_pos=(1 << 32) + 1), "FT_ERR_SHAPE")):
            assert call(rot=rotation(**kw)) == want, kw
        for eps in (-1.0, math.nan, math.inf):
            assert call(eps=eps) == "FT_ERR_INVALID_ARG"
        assert call(t=-1) == "FT_ERR_INVALID_ARG"
        assert call(t=0) == "FT_OK"
    assert status("ft_rope", None, 0, FAKE, 256, 64, 2, 4, 64, None, 0.0, FAKE, 256, 64, None) == "FT_ERR_INVALID_ARG"
    for kw, want in ((dict(dim=1), "FT_ERR_SHAPE"), (dict(dim=514), "FT_ERR_SHAPE"), (dict(heads=-1), "FT_ERR_INVALID_ARG"), (dict(heads=1025), "FT_ERR_SHAPE"),
                     (dict(t=(1 << 24) + 1), "FT_ERR_SHAPE"), (dict(t=1 << 24, heads=65, xt=65 * 64, ot=65 * 64), "FT_ERR_SHAPE"), (dict(xt=63), "FT_ERR_INVALID_ARG"),
                     (dict(xh=63), "FT_ERR_INVALID_ARG"), (dict(xt=BIG), "FT_ERR_INVALID_ARG"), (dict(oh=-64), "FT_ERR_INVALID_ARG"), (dict(x=None), "FT_ERR_INVALID_ARG"),
                     (dict(out=None), "FT_ERR_INVALID_ARG"), (dict(x=ODD), "FT_ERR_ALIGNMENT"), (dict(out=ODD), "FT_ERR_ALIGNMENT"), (dict(weight=ODD), "FT_ERR_ALIGNMENT"),
                     (dict(out=FAKE, ot=512), "FT_ERR_INVALID_ARG"), (dict(heads=0), "FT_OK")):
        assert rope(**kw) == want, kw


def test_store_refused():
    assert store(cache(k_type=2)) == "FT_ERR_UNSUPPORTED"
    assert store(cache(head_dim=80)) == "FT_ERR_SHAPE"
    for kw, want in ((dict(n_head=-1), "FT_ERR_INVALID_ARG"), (dict(n_head=1025), "FT_ERR_SHAPE"), (dict(q=None), "FT_ERR_INVALID_ARG"), (dict(q_out=None), "FT_ERR_INVALID_ARG"),
                     (dict(k=None), "FT_ERR_INVALID_ARG"), (dict(v=None), "FT_ERR_INVALID_ARG"), (dict(slots=None), "FT_ERR_INVALID_ARG"), (dict(q=ODD), "FT_ERR_ALIGNMENT"),
                     (dict(q_out=ODD), "FT_ERR_ALIGNMENT"), (dict(k=ODD), "FT_ERR_ALIGNMENT"), (dict(v=ODD), "FT_ERR_ALIGNMENT"), (dict(slots=FAKE + 4), "FT_ERR_ALIGNMENT"),
                     (dict(k_weight=ODD), "FT_ERR_ALIGNMENT"), (dict(q_weight=ODD), "FT_ERR_ALIGNMENT"), (dict(k_token=63), "FT_ERR_INVALID_ARG"),
                     (dict(v_head=BIG), "FT_ERR_INVALID_ARG"), (dict(q_head=1), "FT_ERR_INVALID_ARG"), (dict(out_token=63), "FT_ERR_INVALID_ARG"),
                     (dict(q_out=FAKE, out_token=512), "FT_ERR_INVALID_ARG"), (dict(t=(1 << 24) + 1), "FT_ERR_SHAPE")):
        assert store(**kw) == want, kw
    assert status("ft_kv_store_rope", ctypes.byref(cache()), rotation(), 0, None, FAKE, 2, None) == "FT_ERR_INVALID_ARG"


def test_table_refused():
    def table(freqs=FAKE, half=64, n_pos=10, out=FAKE):
        return status("ft_rope_table", freqs, half, n_pos, 1.0, out, None)

    for kw, want in ((dict(half=0), "FT_ERR_INVALID_ARG"), (dict(n_pos=-1), "FT_ERR_INVALID_ARG"), (dict(half=(1 << 15) + 1), "FT_ERR_SHAPE"),
                     (dict(n_pos=(1 << 24) + 1), "FT_ERR_SHAPE"), (dict(freqs=None), "FT_ERR_INVALID_ARG"), (dict(out=None), "FT_ERR_INVALID_ARG"),
                     (dict(freqs=FAKE + 4), "FT_ERR_ALIGNMENT"), (dict(out=ODD), "FT_ERR_ALIGNMENT"), (dict(n_pos=0), "FT_OK")):
        assert table(**kw) == want, kw


def test_norm_refused():
    assert status("ft_norm", 0, FAKE, 64, 2, 64, None, None) == "FT_ERR_INVALID_ARG"
    for kw, want in ((dict(ty=3), "FT_ERR_UNSUPPORTED"), (dict(rows=-1), "FT_ERR_INVALID_ARG"), (dict(width=0), "FT_ERR_INVALID_ARG"),
                     (dict(width=32769, ldx=32769, ld_out=32769), "FT_ERR_SHAPE"), (dict(rows=(1 << 24) + 1), "FT_ERR_SHAPE"), (dict(out=None), "FT_ERR_INVALID_ARG"),
                     (dict(x=None), "FT_ERR_INVALID_ARG"), (dict(ldx=63), "FT_ERR_INVALID_ARG"), (dict(ld_out=63), "FT_ERR_INVALID_ARG"), (dict(ldx=BIG), "FT_ERR_INVALID_ARG"),
                     (dict(residual=FAKE, ld_residual=63), "FT_ERR_INVALID_ARG"), (dict(gate=FAKE, ld_gate=63), "FT_ERR_INVALID_ARG"),
                     (dict(gate=FAKE, ld_gate=-64), "FT_ERR_INVALID_ARG"), (dict(r=FAKE + 4096, ld_r=0), "FT_ERR_INVALID_ARG"), (dict(r=FAKE, ld_r=64), "FT_ERR_INVALID_ARG"),
                     (dict(ld_out=128), "FT_ERR_INVALID_ARG"), (dict(x=FAKE + 4096, residual=FAKE, ld_residual=128), "FT_ERR_INVALID_ARG"),
                     (dict(post_weight=FAKE), "FT_ERR_INVALID_ARG"), (dict(post_bias=FAKE), "FT_ERR_INVALID_ARG"), (dict(eps=-1e-9), "FT_ERR_INVALID_ARG"),
                     (dict(eps=math.nan), "FT_ERR_INVALID_ARG"), (dict(scale=math.inf), "FT_ERR_INVALID_ARG"), (dict(x=ODD), "FT_ERR_ALIGNMENT"),
                     (dict(gate=ODD), "FT_ERR_ALIGNMENT"), (dict(weight=ODD), "FT_ERR_ALIGNMENT"), (dict(xq=FAKE + 8, act=6), "FT_ERR_ALIGNMENT"),
                     (dict(xq=FAKE, act=2), "FT_ERR_UNSUPPORTED"), (dict(xq=FAKE, act=7), "FT_ERR_SHAPE"),
                     (dict(xq=FAKE, act=6, width=40, ldx=40, ld_out=40), "FT_ERR_SHAPE"), (dict(rows=0), "FT_OK")):
        assert norm(**kw) == want, kw


def test_lora_refused():
    for kw, want in ((dict(tx=3), "FT_ERR_UNSUPPORTED"), (dict(tw=-1), "FT_ERR_UNSUPPORTED"), (dict(t=-1), "FT_ERR_INVALID_ARG"), (dict(k=0), "FT_ERR_INVALID_ARG"),
                     (dict(many=0), "FT_ERR_INVALID_ARG"), (dict(rank=0), "FT_ERR_INVALID_ARG"), (dict(rank=257), "FT_ERR_SHAPE"), (dict(many=8193), "FT_ERR_SHAPE"),
                     (dict(t=(1 << 20) + 1), "FT_ERR_SHAPE"), (dict(k=(1 << 20) + 1, ldx=1 << 21), "FT_ERR_SHAPE"),
                     (dict(n=(1 << 20) + 1, ldy=1 << 21, ldo=1 << 21), "FT_ERR_SHAPE"), (dict(ldx=63), "FT_ERR_INVALID_ARG"), (dict(ldy=31, out=FAKE + 4096), "FT_ERR_INVALID_ARG"),
                     (dict(ldo=31, out=FAKE + 4096), "FT_ERR_INVALID_ARG"), (dict(ldo=64), "FT_ERR_INVALID_ARG"), (dict(ldx=BIG), "FT_ERR_INVALID_ARG"),
                     (dict(x=None), "FT_ERR_INVALID_ARG"), (dict(a=None), "FT_ERR_INVALID_ARG"), (dict(b=None), "FT_ERR_INVALID_ARG"), (dict(ids=None), "FT_ERR_INVALID_ARG"),
                     (dict(out=None), "FT_ERR_INVALID_ARG"), (dict(x=ODD), "FT_ERR_ALIGNMENT"), (dict(a=FAKE + 1), "FT_ERR_ALIGNMENT"), (dict(ids=ODD), "FT_ERR_ALIGNMENT"),
                     (dict(y=ODD, out=FAKE), "FT_ERR_ALIGNMENT"), (dict(ranks=ODD), "FT_ERR_ALIGNMENT"), (dict(scales=ODD), "FT_ERR_ALIGNMENT"),
                     (dict(workspace=FAKE + 8, workspace_bytes=1 << 30), "FT_ERR_ALIGNMENT"), (dict(workspace=FAKE, workspace_bytes=16), "FT_ERR_NO_SCRATCH"),
                     (dict(t=0), "FT_OK"), (dict(n=0), "FT_OK")):
        assert lora(**kw) == want, kw


def test_adapter_scratch_sizes():
    """A size holds for every smaller number of tokens."""
    for k, many, rank in ((4096, 8, 16), (100, 1, 256), (14336, 300, 64)):
        last = 0
        for t in list(range(1, 200)) + [255, 256, 257, 1000, 1024, 5000, 32768, 40000, 1 << 20]:
            n = ft.lora_scratch_bytes(t, k, many, rank)
            assert n >= last, (t, n, last)
            last = n
    for bad in ((0, 64, 1, 1), (1, 0, 1, 1), (1, 64, 0, 1), (1, 64, 1, 257), (1 << 21, 64, 1, 1)):
        assert ft.lib().ft_lora_scratch_bytes(*bad) == 0
        with pytest.raises(ft.FtError):
            ft.lora_scratch_bytes(*bad)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        ft.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(10, 64))
    with pytest.raises(ValueError):
        ft.norm(x[0])
    with pytest.raises(ValueError):
        ft.lora(x[0], torch.zeros(1, 4, 64), torch.zeros(1, 8, 4), torch.zeros(4, dtype=torch.int32))
    for call in (lambda: ft.rope([1.0], None, None), lambda: ft.norm(None), lambda: ft.lora(x[0], None, None, None),
                 lambda: ft.norm(x[0], eps="1")):
        with pytest.raises((TypeError, ValueError)):
            call()
    for kw in (dict(kind="mean"), dict(act="Q4_0")):
        with pytest.raises(ValueError):
            ft.norm(x[0], **kw)


def test_angles():
    f, s = ft.rope_freqs(8, 10000.0)
    assert s == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001])
    assert ft.rope_freqs(8, 10000.0, "linear", 4.0)[0] == pytest.approx([x / 4 for x in f])
    n, _ = ft.rope_freqs(8, 10000.0, "ntk", 4.0)
    assert n[0] == 1.0 and n[3] == pytest.approx(0.001 / 4)   # the longest wave stretches by the factor, the shortest not
    # by turns over the original positions: above `high` as they are, below `low` by the factor, linear between
    f, _ = ft.rope_freqs(64, 10000.0)
    b, s = ft.rope_freqs(64, 10000.0, "blend", 8.0, 4096, 1.0, 4.0)
    assert s == 1.0
    for x, y in zip(f, b):
        turns = 4096 * x / (2 * math.pi)
        mix = min(1.0, max(0.0, (turns - 1) / 3))
        assert y == pytest.approx(mix * x + (1 - mix) * x / 8)
    r, s = ft.rope_freqs(64, 10000.0, "ramp", 8.0, 4096)
    assert s == pytest.approx(0.1 * math.log(8) + 1)
    assert r[0] == f[0] and r[-1] == pytest.approx(f[-1] / 8)
    assert all(x / 8 <= y * (1 + 1e-12) and y <= x for x, y in zip(f, r))
    assert ft.rope_freqs(2, 10000.0, "ntk", 4.0) == ([1.0], 1.0)
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0), dict(rot_dim=8, factor=0.0), dict(rot_dim=8, scaling="other"),
                dict(rot_dim=8, scaling="blend", low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            ft.rope_freqs(**bad)
