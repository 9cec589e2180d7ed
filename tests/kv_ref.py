"""Plain 64-bit forms of the cache, the attention over it and the scored router, from
their definitions in include/ft.h, for the tests (numpy; no code of the library)."""
import numpy as np

BLOCK_BYTES = {"Q8_0": 34, "Q4_0": 18}


def quantize(x, ty):
    """x [..., D] float32 -> integer codes [..., D] and float16 scales [..., D / 32]."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    if ty == "Q8_0":
        d = np.abs(b).max(-1) / np.float32(127)
        lo, hi = -127, 127
    else:
        at = np.abs(b).argmax(-1)[..., None]   # the first of equal magnitudes
        d = np.take_along_axis(b, at, -1)[..., 0] / np.float32(-8)
        lo, hi = -8, 7
    d = np.clip(d, -65504, 65504).astype(np.float16)
    d[d == 0] = 0
    df = d.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = (b / df).astype(np.float64)        # the correctly rounded fp32 quotient
    q = np.sign(t) * np.floor(np.abs(t) + 0.5)
    q = np.where(df == 0, 0, np.clip(np.nan_to_num(q, nan=0.0, posinf=1e9, neginf=-1e9), lo, hi))
    return q.astype(np.int64).reshape(x.shape), d


def values(q, d):
    return (q.reshape(*q.shape[:-1], q.shape[-1] // 32, 32) * d.astype(np.float64)[..., None]).reshape(q.shape)


def code_bytes(ty, dim, page):
    return dim * page // (1 if ty == "Q8_0" else 2)


def read_slot(pool, ty, side, page, heads, dim, slot):
    """Codes [heads, dim] and scales [heads, dim / 32] of one slot, byte by byte from the pool."""
    hb = page * (dim // 32) * BLOCK_BYTES[ty]
    raw = np.asarray(pool, np.uint8).reshape(-1, heads, hb)[slot // page]
    j, nb = slot % page, dim // 32
    q = np.empty((heads, dim), np.int64)
    d = np.empty((heads, nb), np.float16)
    for h in range(heads):
        for e in range(dim):
            b, i = divmod(e, 32)
            if side == "v":
                if ty == "Q8_0":
                    q[h, e] = int(raw[h, e * page + j]) - 128
                else:
                    q[h, e] = (int(raw[h, (16 * b + i % 16) * page + j]) >> (4 * (i // 16)) & 15) - 8
            elif ty == "Q8_0":
                m = min(2, nb - b // 2 * 2)
                q[h, e] = int(raw[h, page * 64 * (b // 2) + j * 32 * m + i // 8 * 8 * m + b % 2 * 8 + i % 8]) - 128
            else:
                m = min(4, nb - b // 4 * 4)
                at = page * 64 * (b // 4) + j * 16 * m + i // 8 * 4 * m + b % 4 * 4
                word = int.from_bytes(raw[h, at:at + 4].tobytes(), "little")
                q[h, e] = (word >> (4 * (i % 8 // 2 + 4 * (i % 2))) & 15) - 8
        at = code_bytes(ty, dim, page)
        d[h] = raw[h, at:].view(np.float16).reshape(nb, page)[:, j]
    return q, d


def attention(q, k, v, count, kv_len, scale=None, causal=True, window=0, softcap=0.0, slopes=None, prefix=0):
    """One sequence: q [count, heads, D], k, v [kv_len, kv_heads, D] (float64).  Returns the output and, per (token,
    head), what an error bound needs: the largest sum of |scale q k| over the visible keys, the largest distance bias,
    and sum p |v|."""
    n, heads, dim = q.shape
    group = heads // max(k.shape[1], 1)
    scale = dim ** -0.5 if scale is None else scale
    out = np.zeros((n, heads, dim))
    terms, bias, mass = np.zeros((n, heads)), np.zeros((n, heads)), np.zeros((n, heads, dim))
    for i in range(n):
        pos = kv_len - count + i
        key = np.arange(kv_len)
        seen = key <= pos if causal else key >= 0
        if window:
            seen = seen & (key > pos - window)
        seen = seen | (key < prefix)
        if not seen.any():
            continue
        for h in range(heads):
            kk, vv = k[seen, h // group], v[seen, h // group]
            s = kk @ q[i, h] * scale
            terms[i, h] = np.max(np.abs(kk) @ np.abs(q[i, h])) * abs(scale)
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                far = slopes[h] * np.abs(pos - key[seen])
                s = s - far
                bias[i, h] = np.max(far) + np.max(np.abs(s))
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vv
            mass[i, h] = p @ np.abs(vv)
    return out, terms, bias, mass


def attention_bound(out, terms, bias, mass, v, dtype, softcap=0.0):
    """How far an output may be off.
    score: q as a pair of fp16 (2^-22), 32 products and the blocks' scales summed in fp32 (at most 48 roundings of the
    sum of |terms|), three more factors: (4 + 48 + 3) 2^-24 of the terms; under softcap tanh is within 2^-21 of its
    result, times the cap; a bias takes three roundings of its own size.  p = exp2(score): a score off by x moves p by
    x relative, numerator and denominator both.
    bf16 rows: a key's code times its scale is rounded to fp16 once, 2^-11 of each term.
    exp2 2^-23; p times V's scale: 2^-21 as an fp16 pair (fp32 rows), 2^-11 as one fp16 (fp16 rows); bf16 rows: p rounded
    to fp16, and its product with the scale again, 2 * 2^-11.  Products summed in fp32: at most one
    rounding per key a wave sums, keys / 4 + 64; the joins of waves and splits: 64 roundings more.
    All of it relative to sum p |v|; then the output's own rounding.
    The fp16 numbers p d (d: V's scale) end at 2^-25 absolute.  Their unit 2^-C is such that 2^14 <= 2^C d_max, d_max the
    largest scale of the step that set it, and the sum of p that divides is at least 2^C in it: a code times what is lost
    is 128 * 2^-25 / 2^C <= 2^-32 d_max = 2^-39 v_max per key for Q8_0, 8 * 2^-25 / 2^C = 2^-36 d_max = 2^-39 v_max for Q4_0
    (v_max of all the sequence's keys; d_max = v_max / 127 or / 8 but for the rounding of d: twice that here).
    bf16 rows lose 2^-25 in p (times a scale below 2) and in the product: three times that, under 2^-37 v_max per key; and
    scales are held to 2^-25 of the step's largest, 2^-25 v_max over all keys together."""
    keys = len(v)
    lost = (keys * 2.0 ** -37 + 2.0 ** -25 * (dtype == "bf16")) * (np.abs(v).max() if keys else 0.0)
    eps_k, eps_p, eps_out = {"f32": (0, 2.0 ** -21, 2.0 ** -24), "f16": (0, 2.0 ** -11, 2.0 ** -11),
                             "bf16": (2.0 ** -11, 2 * 2.0 ** -11, 2.0 ** -8)}[dtype]
    score = (eps_k + 55 * 2.0 ** -24) * terms + 3 * 2.0 ** -24 * bias + softcap * 2.0 ** -21
    rel = 2 * np.expm1(score) + 2.0 ** -22 + eps_p + (keys / 2 + 256) * 2.0 ** -24
    return rel[..., None] * mass + eps_out * np.abs(out) + lost + 1e-30


def route(x, topk, sigmoid=False, bias=None, n_group=1, topk_group=None, group_top=1, renorm=True, scale=1.0):
    x = np.asarray(x, np.float64)
    t, e = x.shape
    if sigmoid:
        with np.errstate(over="ignore"):
            score = 1 / (1 + np.exp(-x))
    else:
        ex = np.exp(x - x.max(-1, keepdims=True))
        score = ex / ex.sum(-1, keepdims=True)
    choice = score + (0 if bias is None else np.asarray(bias, np.float64))
    ids, w = np.empty((t, topk), np.int32), np.empty((t, topk))
    size = e // n_group
    for r in range(t):
        c = choice[r].copy()
        if n_group > 1:
            best = [np.sort(c[g * size:(g + 1) * size])[::-1][:group_top].sum() for g in range(n_group)]
            order = sorted(range(n_group), key=lambda g: (-best[g], g))[:topk_group or n_group]
            open_ = np.zeros(e, bool)
            for g in order:
                open_[g * size:(g + 1) * size] = True
            cand = np.flatnonzero(open_)
        else:
            cand = np.arange(e)
        pick = sorted(cand, key=lambda i: (-c[i], i))[:topk]
        ids[r], w[r] = pick, score[r][pick]
        if renorm:
            s = w[r].sum()
            w[r] = w[r] / s if s > 0 else 0
    return ids, w * scale
