"""GPU: the norm around a block against its definition: in 64 bits within the roundings counted, and to the bit in single
fp32 operations; its quantized blocks are the oracle's of its fp32 rows."""
import numpy as np
import pytest
import torch

import oracle
from block_quantized_matvec_amd import ft
from tests import layer_ref as ref
from tests.gpu_util import dev, host, need_gpu, own_stream

pytestmark = pytest.mark.gpu


def lines(rows, width, dtype, seed, scale=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, width + pad, generator=g) * scale).to(ref.DT[dtype]).cuda()[:, :width]


def vector(width, seed, mean=1.0):
    return (mean + 0.3 * np.random.RandomState(seed).randn(width)).astype(np.float32)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(got, x, dtype, eps=1e-6, **o):
    """got: (r, n); o: block's arguments, tensors of dtype or fp32 vectors."""
    args = dict(o, eps=eps)
    for k in ("residual", "gate"):
        args[k] = f64(o.get(k))
    r, n = ref.block(f64(x), **args)
    single = dict(args, residual=None if args["residual"] is None else args["residual"].astype(np.float32),
                  gate=None if args["gate"] is None else args["gate"].astype(np.float32))
    r1, n1 = ref.block(f64(x).astype(np.float32), at=np.float32, **single)
    t = ref.DT[dtype]
    for g, one in zip(got, (r1, n1)):
        if g is not None:   # rounded once from the single operations
            assert torch.allclose(g.cpu(), torch.from_numpy(np.ascontiguousarray(one)).to(t), rtol=0, atol=0, equal_nan=True)
    # 64 bits: r carries a rounding per step of b (norm 3 with its weight, bias, gate, scale) and its own;
    # n one of r per element and of the factor, two products and the bias
    if np.isnan(n).any():   # a row of one value without eps: 0 / 0, in 64 bits too
        assert np.array_equal(np.isnan(f64(got[1])), np.isnan(n))
        return
    with np.errstate(invalid="ignore"):
        b = np.abs(r - (0 if args["residual"] is None else args["residual"]))
        pb = 0.0
        if o.get("post_bias") is not None:
            pb = np.abs(o["post_bias"] * np.abs(args["gate"] if args["gate"] is not None else 1.0) * o.get("scale", 1.0))
        u = 2.0 ** -24 * 1.01
        r_off = u * (7 * (b + 2 * pb) + np.abs(r))
        if got[0] is not None:
            off = np.abs(f64(got[0]) - r)
            assert np.all(off <= r_off + ref.rounding(r, dtype) + 2.0 ** -40), np.max(off)
        if got[1] is not None:
            w = r if o.get("kind", "rms") == "rms" else r - r.mean(-1, keepdims=True)
            f = ref.rstd((w * w).mean(-1, keepdims=True), eps) * np.abs(1.0 if o.get("weight") is None else o["weight"])
            spread = r_off.max(-1, keepdims=True)   # a mean moves by no more; the factor by the rows' relative error
            rel = np.sqrt((r_off ** 2).mean(-1, keepdims=True)) * ref.rstd((w * w).mean(-1, keepdims=True), eps)
            bias = np.abs(0.0 if o.get("bias") is None else o["bias"])
            n_off = f * (r_off + (spread if o.get("kind") == "layer" else 0)) + (2 * rel + 5 * u) * np.abs(w) * f + u * (bias + np.abs(n))
            off = np.abs(f64(got[1]) - n)
            assert np.all(off <= n_off + ref.rounding(n, dtype) + 2.0 ** -40), np.max(off / (n_off + 2.0 ** -40))


WIDTHS = [1, 5, 8, 32, 100, 255, 512, 513, 1536, 2048, 2056, 4096, 4100, 5002, 8192, 8200, 16384, 16390, 32768]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, kind):
    need_gpu()
    w, b = vector(width, 1), vector(width, 2, 0.0)
    for dtype, rows in (("f32", 5), ("f16", 1), ("bf16", 3)):
        x, res = lines(rows, width, dtype, 3), lines(rows, width, dtype, 4, 2.0)
        r, n, xq = ft.norm(x, weight=dev(w), bias=dev(b), residual=res, kind=kind, eps=1e-5)
        assert xq is None
        check((r, n), x, dtype, 1e-5, kind=kind, weight=w, bias=b, residual=res)
        r, n, _ = ft.norm(x, kind=kind, eps=1e-5)
        assert r is x
        check((None, n), x, dtype, 1e-5, kind=kind)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", ["none", "plain", "weight", "both"])
@pytest.mark.parametrize("gate", ["none", "vector", "line", "rows"])
def test_steps(kind, post, gate, dtype):
    need_gpu()
    for rows, width, pad, scale, residual in ((1, 2048, 0, 1.0, True), (9, 520, 3, 0.25, False), (6, 4096, 8, 1.5, True)):
        x = lines(rows, width, dtype, 5, 3.0, pad)
        res = lines(rows, width, dtype, 6, 1.0, pad) if residual else None
        g = {"none": None, "vector": lines(1, width, dtype, 7)[0], "line": lines(1, width, dtype, 7), "rows": lines(rows, width, dtype, 7, 1.0, pad)}[gate]
        pw, pb = vector(width, 8) if post in ("weight", "both") else None, vector(width, 9, 0.0) if post == "both" else None
        w = vector(width, 10)
        r, n, _ = ft.norm(x, weight=dev(w), residual=res, post=True if post == "plain" else None, post_weight=None if pw is None else dev(pw),
                          post_bias=None if pb is None else dev(pb), gate=g, scale=scale, kind=kind)
        if r is x:
            r = None
        check((r, n), x, dtype, kind=kind, post=post != "none", post_weight=pw, post_bias=pb, gate=g, scale=scale, residual=res, weight=w)


@pytest.mark.parametrize("act", ["Q8_1", "Q8_0", "Q8_K"])
@pytest.mark.parametrize("width", [256, 512, 1024, 2048, 4096, 7168, 8192, 14336, 32768])
def test_blocks(width, act):
    need_gpu()
    for dtype, rows, kind in (("f32", 1, "rms"), ("f32", 7, "layer"), ("bf16", 4, "rms")):
        x, res, w = lines(rows, width, dtype, 11), lines(rows, width, dtype, 12), vector(width, 13)
        x[:, 64:96] = res[:, 64:96] = 0   # a block of zeros (not under a mean)
        r, n, xq = ft.norm(x, weight=dev(w), residual=res, act=act, kind=kind)
        assert n is None
        r1, n1 = ref.block(f64(x).astype(np.float32), residual=f64(res).astype(np.float32), weight=w, eps=1e-6, kind=kind, at=np.float32)
        assert np.array_equal(host(xq), oracle.quantize(act, n1))
        _, n, again = ft.norm(x, weight=dev(w), residual=res, act=act, kind=kind, rows=True)
        assert torch.equal(xq, again)
        check((r, n), x, dtype, kind=kind, residual=res, weight=w)


def test_blocks_of_32():
    need_gpu()
    x = lines(5, 96, "f32", 14)
    for act in ("Q8_1", "Q8_0"):
        _, _, xq = ft.norm(x, act=act)
        assert np.array_equal(host(xq), oracle.quantize(act, ref.norm(f64(x).astype(np.float32), eps=1e-6, at=np.float32)))


def test_in_place():
    need_gpu()
    for width in (512, 1000, 4096):
        x, res, w = lines(6, width, "f32", 15), lines(6, width, "f32", 16), vector(width, 17)
        want = ft.norm(x, weight=dev(w), residual=res, scale=0.5)
        a, b = x.clone(), res.clone()
        r, n, _ = ft.norm(a, weight=dev(w), residual=b, scale=0.5, r=b, out=a)
        assert r is b and n is a
        assert torch.equal(a, want[1]) and torch.equal(b, want[0])
        a, b = x.clone(), res.clone()
        ft.norm(a, weight=dev(w), residual=b, scale=0.5, r=a, out=b)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_only_the_stream():
    """After a last block there is no norm: r alone."""
    need_gpu()
    x, res, pw = lines(4, 768, "bf16", 18), lines(4, 768, "bf16", 19), vector(768, 20)
    r, n, xq = ft.norm(x, residual=res, post_weight=dev(pw), rows=False)
    assert n is None and xq is None
    check((r, None), x, "bf16", residual=res, post=True, post_weight=pw)


def test_rows_keep_to_themselves():
    need_gpu()
    for width in (96, 1000, 4096):
        x = lines(5, width, "f32", 21)
        want = ft.norm(x)[1].clone()
        x[1, 3], x[3, 7] = float("nan"), float("inf")
        n = ft.norm(x)[1]
        assert torch.equal(n[[0, 2, 4]], want[[0, 2, 4]])
        assert torch.isnan(n[1]).all() and torch.isnan(n[3, 7])
        assert ft.norm(x, out=torch.empty(5, width, device="cuda"))[1].shape == (5, width)
    assert ft.norm(lines(0, 64, "f32", 1))[1].shape == (0, 64)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_far_values(kind):
    """Squares past fp32, means far above the deviations, deviations near fp32's end, rows of one value."""
    need_gpu()
    width = 1024
    base = lines(4, width, "f32", 22)
    for x in (base * 1e30, base * 1e-30, base + 1e4, base * 1e-3 + 1e5, base * 0.1 + 1e5):
        check((None, ft.norm(x, kind=kind, eps=0.0)[1]), x, "f32", 0.0, kind=kind)
    flat = torch.full((2, width), 3.7, device="cuda")
    n = host(ft.norm(flat, kind=kind, eps=1e-6)[1])
    if kind == "layer":
        assert np.all(np.abs(n) <= 1e3 * 2.0 ** -50 * 3.7)   # the 64-bit mean's rounding over 1e-3
    else:
        assert np.all(np.abs(n - 1) <= 1e-6)
    assert torch.all(ft.norm(torch.zeros(2, width, device="cuda"), kind=kind)[1] == 0)


def test_many_rows():
    need_gpu()
    for rows, width in ((70001, 40), (3001, 2048)):
        x, res = lines(rows, width, "bf16", 23), lines(rows, width, "bf16", 24)
        w = vector(width, 25)
        r, n, _ = ft.norm(x, weight=dev(w), residual=res)
        check((r, n), x, "bf16", residual=res, weight=w)


def test_captured():
    need_gpu()
    x, res, w = lines(3, 4096, "f32", 26), lines(3, 4096, "f32", 27), dev(vector(4096, 28))
    r, xq = torch.empty_like(res), torch.empty(3, ft.row_bytes("Q8_1", 4096), dtype=torch.uint8, device="cuda")
    s, graph = own_stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        ft.norm(x, weight=w, residual=res, act="Q8_1", r=r, xq=xq, stream=s)
    for i in range(3):
        x.copy_(lines(3, 4096, "f32", 30 + i))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ft.norm(x, weight=w, residual=res, act="Q8_1")
        assert torch.equal(r, want[0]) and torch.equal(xq, want[2])
