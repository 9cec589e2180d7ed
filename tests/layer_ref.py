"""Plain forms of the operators around the quantized products (rotary positions, norms, adapters) from their definitions
in include/ft.h, for the tests (numpy; no code of the library): in 64 bits, and in single fp32 operations where the
header fixes every rounding."""
import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}


def rounding(value, dtype):
    """At most half a step: relative to the value, and below the type's normal numbers (fp16: 2^-14, steps of 2^-24) absolute."""
    return np.maximum(HALF_STEP[dtype] * np.abs(value) * 1.01, torch.finfo(DT[dtype]).smallest_normal * HALF_STEP[dtype] * 1.01)


def table(n_pos, freqs, scale=1.0):
    a = np.arange(n_pos, dtype=np.float64)[:, None] * np.asarray(freqs, np.float64)
    return np.concatenate([np.cos(a) * scale, np.sin(a) * scale], 1)


def rstd(mean_square, eps):
    with np.errstate(divide="ignore", invalid="ignore"):
        return 1.0 / np.sqrt(mean_square + eps)


def pairs(dim, rot, interleaved):
    """Indices of every pair's two elements."""
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def turn(x, pos, tab, interleaved, weight=None, eps=0.0, kind=np.float64):
    """x [t, heads, dim] turned by rows of tab at pos, in `kind` (float32: single operations, as the library's)."""
    rot = tab.shape[1]
    x = np.asarray(x, kind).copy()
    if weight is not None:
        r = rstd(np.mean(np.asarray(x, np.float64) ** 2, -1, keepdims=True), eps).astype(kind)
        x = x * r * np.asarray(weight, kind)
    row = np.asarray(tab, kind)[np.clip(pos, 0, tab.shape[0] - 1)][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    i, j = pairs(x.shape[-1], rot, interleaved)
    a, b = x[..., i], x[..., j]
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


def norm(x, kind="rms", eps=0.0, weight=None, bias=None, at=np.float64):
    w = np.asarray(x, np.float64)
    if kind == "layer":
        w = w - w.mean(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        n = w.astype(at) * rstd((w * w).mean(-1, keepdims=True), eps).astype(at)
    if weight is not None:
        n = n * np.asarray(weight, at)
    if bias is not None:
        n = n + np.asarray(bias, at)
    return n


def block(x, residual=None, post=False, post_weight=None, post_bias=None, gate=None, scale=1.0, kind="rms", eps=0.0, weight=None,
          bias=None, at=np.float64):
    """(r, n) of ft_norm."""
    b = np.asarray(x, at)
    if post:
        b = norm(b, kind, eps, post_weight, post_bias, at)
    if gate is not None:
        b = b * np.asarray(gate, at)
    b = b * at(scale)
    r = b if residual is None else np.asarray(residual, at) + b
    return r, norm(r, kind, eps, weight, bias, at)


def lora(x, a, b, ids, y=None, scales=None, ranks=None):
    """(out, bound of its rounding): sums of k, then of rank products in fp32, each operand good to 2^-23."""
    t, k = x.shape
    many, rank = a.shape[:2]
    n = b.shape[1]
    out = np.zeros((t, n)) if y is None else y.astype(np.float64).copy()
    u = 2.0 ** -24
    off = u * np.abs(out)
    for i in range(t):
        e = int(ids[i])
        if not 0 <= e < many:
            continue
        r = rank if ranks is None else max(0, min(rank, int(ranks[e])))
        A, B, s = a[e, :r].astype(np.float64), b[e, :, :r].astype(np.float64), 1.0 if scales is None else float(scales[e])
        h = A @ x[i].astype(np.float64)
        gap = (k + 24) * u * (np.abs(A) @ np.abs(x[i].astype(np.float64)))
        add = s * (B @ h)
        out[i] += add
        off[i] += abs(s) * (np.abs(B) @ (gap + (r + 8) * u * (np.abs(h) + gap))) + 2 * u * np.abs(out[i])
    return out, off
