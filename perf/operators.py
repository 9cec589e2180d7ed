"""The decoder-layer operators around the quantized products, case by case: the paged
block-quantized key/value cache (written and read back), attention that reads it (single
tokens, prompts, a prefix shared by the batch) and the router of a mixture of experts.

``own`` chooses between the operators in plain torch operations and the library's calls;
``prepare`` makes the same inputs for both.

Cache pages (``include/ft.h`` holds the same definition).  A pool is [n_pages][n_kv_head]
page heads; a page head of P keys, D elements each (NB = D / 32 blocks), is its codes and
then its scales, fp16 [NB][P].  Element e = 32 b + i of key j has its code
  K, Q8_0: at P * 64 * (b / 2) + j * 32 m + (i / 8) * 8 m + (b % 2) * 8 + i % 8, with m = the
           blocks in group b / 2 (2, or 1 in a last odd group); the byte is the code + 128;
  K, Q4_0: in the 32-bit word at P * 64 * (b / 4) + j * 16 m + (i / 8) * 4 m + (b % 4) * 4, m = the
           blocks in group b / 4 (4 or what is left); nibble (i % 8) / 2 + 4 * (i % 2); code + 8;
  V, Q8_0: at e * P + j; the byte is the code + 128;
  V, Q4_0: at (16 b + i % 16) * P + j, low nibble for i < 16 and high above; code + 8.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK_BYTES = {"Q8_0": 34, "Q4_0": 18}
MASKED = float("-inf")


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attn(name, **kw):
    case = dict(name=name, op="attn", n_seq=1, new=1, new_max=1, kv=1024, kv_max=1024, idle=0, heads=32, kv_heads=8, dim=128,
                page=64, k="Q8_0", v="Q8_0", dtype="f32", causal=True, window=0, sinks=0, softcap=0.0, alibi=False, shared=0)
    case.update(kw)
    return case


def listed():
    return [
        # one decode step of a small batch: the new tokens' rows, as the fused q/k/v product left them
        dict(name="cache_step", op="cache", tokens=8, heads=8, dim=128, page=16, k="Q8_0", v="Q8_0", dtype="f32", pad=4096, skip=1),
        # a prompt's keys and values written in one go, then read back for reuse elsewhere
        dict(name="cache_prompt", op="cache", tokens=8192, heads=8, dim=128, page=64, k="Q8_0", v="Q4_0", dtype="bf16", pad=0, skip=0),
        # one user, a short context: latency
        _attn("attn_one", kv=777, kv_max=777, page=16),
        # a serving batch of ragged contexts, one of its slots idle
        _attn("attn_batch", n_seq=32, kv=512, kv_max=8192, idle=1),
        # two users deep in a long document
        _attn("attn_long", n_seq=2, kv=100000, kv_max=131071, v="Q4_0", dtype="f16", heads=40, page=128),
        # drafted tokens checked in one pass: window, sink tokens and a bias by distance
        _attn("attn_draft", n_seq=16, new=3, new_max=6, kv=700, kv_max=5000, heads=20, kv_heads=4, dim=64, k="Q4_0", v="Q4_0",
              dtype="bf16", window=1024, sinks=4, alibi=True, page=32),
        # ragged prompts in one batch, scores capped
        _attn("attn_prompt", n_seq=3, new=500, new_max=4096, kv=500, kv_max=4096, dtype="bf16", softcap=50.0),
        # a chunk of a long prompt in full precision
        _attn("attn_chunk", new=1000, new_max=1000, kv=7000, kv_max=7000),
        # few requests that share a system prompt
        _attn("shared_few", n_seq=8, kv=2100, kv_max=2300, shared=2048),
        # many samples of one long context
        _attn("shared_many", n_seq=64, kv=16400, kv_max=16900, shared=16384, dtype="f16"),
        # the router of one decode step
        dict(name="route_step", op="route", tokens=3, experts=128, topk=8, score="softmax", bias=False, groups=1, keep=1, top=1,
             renorm=True, scale=1.0, dtype="f32"),
        # the router of a prompt: sigmoid scores, a balance bias and groups
        dict(name="route_prompt", op="route", tokens=16384, experts=256, topk=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5)))


def draw(rng):
    kind = rng.choice(["cache", "step", "step", "prompt", "shared", "route"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8 if groups < 8 else 4, 1024 // groups)
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(16, experts // groups * keep))
        return dict(op="route", tokens=_log(rng, 1, 16384), experts=experts, topk=topk, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=dtype)
    dim, page = rng.choice([64, 96, 128, 256]), rng.choice([16, 32, 64, 128])
    k = rng.choice(["Q8_0", "Q4_0"])
    v = rng.choice(["Q8_0", "Q4_0"])
    if kind == "cache":
        return dict(op="cache", tokens=_log(rng, 1, 8192), heads=rng.randint(1, 16), dim=dim, page=page, k=k, v=v, dtype=dtype,
                    pad=rng.choice([0, 7, 4096]), skip=rng.choice([0, 0, 3]))
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.randint(1, 32 // kv_heads if kv_heads > 1 else 12)
    case = _attn("", heads=heads, kv_heads=kv_heads, dim=dim, page=page, k=k, v=v, dtype=dtype)
    del case["name"]
    if kind == "step":
        n_seq = _log(rng, 1, 64)
        kv_max = _log(rng, 1, min(131072, 262144 // n_seq))
        case.update(n_seq=n_seq, kv=_log(rng, 1, kv_max), kv_max=kv_max, new_max=rng.choice([1, 1, 1, 2, 5]), idle=rng.choice([0, 0, 1]) if n_seq > 1 else 0)
        if rng.random() < 0.3:
            case.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 4, 70]))
    elif kind == "prompt":
        n_seq = rng.randint(1, 3)
        new_max = _log(rng, 2, 2048)
        new = _log(rng, 1, new_max)
        case.update(n_seq=n_seq, new=new, new_max=new_max, kv=new_max, kv_max=new_max + _log(rng, 1, 2048))
        if rng.random() < 0.3:
            case.update(window=_log(rng, 1, 1024))
        if rng.random() < 0.2:
            case.update(causal=False)
    else:
        n_seq = _log(rng, 2, 64)
        shared = page * max(1, _log(rng, 128, 16384) // page)
        case.update(n_seq=n_seq, shared=shared, kv=shared + 1, kv_max=shared + _log(rng, 1, 512))
    if rng.random() < 0.25:
        case.update(softcap=30.0)
    if rng.random() < 0.25:
        case.update(alibi=True)
    return case


def _lengths(case):
    """Keys and new tokens of every sequence: of the case alone, so that work() knows them."""
    r = random.Random("%(n_seq)d %(kv)d %(kv_max)d %(new)d %(new_max)d" % case)
    n = case["n_seq"]
    kv = [r.randint(case["kv"], case["kv_max"]) for _ in range(n)]
    kv[0] = case["kv_max"]
    new = [r.randint(case["new"], case["new_max"]) for _ in range(n)]
    new[0] = case["new_max"]
    new = [min(a, b) for a, b in zip(new, kv)]
    for i in range(case["idle"]):
        kv[n - 1 - i], new[n - 1 - i] = 0, 1
    return kv, new


def _visible(case, kv, new):
    """Visible (query, key) pairs of one sequence."""
    pairs = 0
    for i in range(new):
        pos = kv - new + i
        last = pos if case["causal"] else kv - 1
        first = max(0, pos - case["window"] + 1) if case["window"] else 0
        pairs += max(0, last - first + 1)
        sinks = min(case["sinks"], kv)
        pairs += sinks - max(0, min(sinks, last + 1) - first)
    return pairs


def work(case):
    if case["op"] == "cache":
        n = case["tokens"] * case["heads"] * case["dim"]
        size = DTYPES[case["dtype"]].itemsize
        held = n // 32 * (BLOCK_BYTES[case["k"]] + BLOCK_BYTES[case["v"]])
        return {"bytes": 2 * n * size * 2 + 2 * held, "flops": 8.0 * n}
    if case["op"] == "route":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * DTYPES[case["dtype"]].itemsize + case["tokens"] * case["topk"] * 8, "flops": 10.0 * n}
    kv, new = _lengths(case)
    size, dim = DTYPES[case["dtype"]].itemsize, case["dim"]
    row = case["kv_heads"] * (dim // 32) * (BLOCK_BYTES[case["k"]] + BLOCK_BYTES[case["v"]])
    reach = case["window"] + max(new) + case["sinks"] if case["window"] else max(kv)
    keys = sum(max(0, min(a, reach) - case["shared"]) for a in kv) + case["shared"]
    pairs = sum(_visible(case, a, b) for a, b in zip(kv, new))
    return {"bytes": keys * row + 2 * sum(new) * case["heads"] * dim * size, "flops": 4.0 * pairs * case["heads"] * dim}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed) * 2654435761 % (1 << 31))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=_device())


def _quantize(x, ty):
    """Codes and fp16 scales of blocks of 32 along the last axis, as the cache holds them."""
    b = x.float().unflatten(-1, (-1, 32))
    if ty == "Q8_0":
        d = (b.abs().amax(-1) / 127).clamp(max=65504.0).half()
        low, high = -127, 127
    else:
        at = b.abs().argmax(-1, keepdim=True)
        d = (b.gather(-1, at).squeeze(-1) / -8).clamp(-65504.0, 65504.0).half()
        low, high = -8, 7
    t = b / d.float().unsqueeze(-1)
    q = t.trunc()
    q = q + torch.where((t - q).abs() >= 0.5, t.sign(), torch.zeros_like(t))
    q = torch.where(d.unsqueeze(-1) == 0, torch.zeros_like(q), q.clamp(low, high))
    return q.to(torch.int16).flatten(-2), torch.where(d == 0, torch.zeros_like(d), d)


def _at(ty, side, dim, page):
    """Byte and shift of every (key, element)'s code in a page head, as the module's text has them."""
    e, j = torch.arange(dim).view(1, -1), torch.arange(page).view(-1, 1)
    b, i, nb = e // 32, e % 32, dim // 32
    if side == "v":
        return (e * page + j, 0 * (e + j)) if ty == "Q8_0" else ((16 * b + i % 16) * page + j, 4 * (i // 16) + 0 * j)
    if ty == "Q8_0":
        m = (nb - b // 2 * 2).clamp(max=2)
        return page * 64 * (b // 2) + j * 32 * m + i // 8 * 8 * m + b % 2 * 8 + i % 8, 0 * (e + j)
    m = (nb - b // 4 * 4).clamp(max=4)
    nibble = i % 8 // 2 + 4 * (i % 2)
    return page * 64 * (b // 4) + j * 16 * m + i // 8 * 4 * m + b % 4 * 4 + nibble // 2, 4 * (nibble % 2) + 0 * j


def _page_head_bytes(ty, dim, page):
    return page * (dim // 32) * BLOCK_BYTES[ty]


def _pack(codes, scales, ty, side):
    """codes [..., page, dim], scales [..., page, dim / 32] -> page heads, uint8 [..., bytes]."""
    *lead, page, dim = codes.shape
    at, shift = _at(ty, side, dim, page)
    at, shift = at.to(codes.device).flatten(), shift.to(codes.device).flatten()
    n = page * dim // (1 if ty == "Q8_0" else 2)
    flat = codes.reshape(-1, page * dim).int() + (128 if ty == "Q8_0" else 8)
    out = torch.zeros(flat.shape[0], n, dtype=torch.int32, device=codes.device)
    out.index_add_(1, at, flat << shift.int())
    held = scales.reshape(-1, page, dim // 32).transpose(1, 2).contiguous().view(torch.uint8).flatten(1)
    return torch.cat([out.to(torch.uint8), held], 1).view(*lead, -1)


def _cache_inputs(case, seed):
    g = _generator(seed)
    t, h, dim, page = case["tokens"], case["heads"], case["dim"], case["page"]
    width = h * dim
    # keys and values are columns of a wider row where `pad` says so: the strides of a fused product
    row = _normal(g, t, case["pad"] + 2 * width)
    row[:, case["pad"]:case["pad"] + width].view(t, h, dim)[..., ::16] *= 6.0  # some of the keys' channels are large
    if t > 1:
        row[t // 2, case["pad"] + width:] = 0.0  # a token whose values are all zero
    row = row.to(DTYPES[case["dtype"]])
    k = row[:, case["pad"]:case["pad"] + width].unflatten(1, (h, dim))
    v = row[:, case["pad"] + width:].unflatten(1, (h, dim))
    n_pages = -(-t // page) + 3
    pages = torch.randperm(n_pages, generator=g, device=_device())
    j = torch.arange(t, device=_device()) + page // 2  # the sequence goes on in the middle of a page
    slots = pages[j // page] * page + j % page
    if case["skip"] and t > 1:
        slots[-case["skip"]:] = -1  # padding behind the batch
    return k, v, slots, n_pages


def _attn_inputs(case, seed):
    g = _generator(seed)
    kv, new = _lengths(case)
    n, page, dim, hk = case["n_seq"], case["page"], case["dim"], case["kv_heads"]
    cols = max(1, -(-max(kv) // page))
    held = case["shared"] // page
    need = [max(0, -(-a // page) - held) for a in kv]
    n_pages = held + sum(need) + 2
    order = torch.randperm(n_pages, generator=g, device=_device())
    table = torch.zeros(n, cols, dtype=torch.int64)
    first = held
    for i, c in enumerate(need):
        table[i, :held] = torch.arange(held)
        table[i, held:held + c] = torch.arange(first, first + c)
        first += c
    table = order[table.to(_device())].int()
    k = _normal(g, n_pages, hk, page, dim)
    k[..., ::16] *= 3.0  # some of the keys' channels are large
    kq, kd = _quantize(k, case["k"])
    del k
    v = _normal(g, n_pages, hk, page, dim)
    v *= torch.exp(0.5 * _normal(g, n_pages, hk, page, 1))  # values of unlike size
    vq, vd = _quantize(v, case["v"])
    del v
    total = sum(new)
    q = _normal(g, total, case["heads"], dim).to(DTYPES[case["dtype"]])
    start = [0]
    for c in new:
        start.append(start[-1] + c)
    slopes = torch.exp2(-8.0 * torch.arange(1, case["heads"] + 1, device=_device()) / case["heads"]) if case["alibi"] else None
    ints = dict(dtype=torch.int32, device=_device())
    return dict(kq=kq, kd=kd, vq=vq, vd=vd, q=q, table=table, kv=torch.tensor(kv, **ints), start=torch.tensor(start, **ints), slopes=slopes,
                sinks=torch.full((n,), case["sinks"], **ints) if case["sinks"] else None)


def _route_inputs(case, seed):
    g = _generator(seed)
    logits = (1.5 * _normal(g, case["tokens"], case["experts"])).to(DTYPES[case["dtype"]])
    logits[:, case["experts"] // 2] = logits[:, 0]  # ties
    bias = 0.1 * _normal(g, case["experts"]) if case["bias"] else None
    return logits, bias


def prepare(case, seed):
    s = dict(case=case)
    if case["op"] == "route":
        s["logits"], s["bias"] = _route_inputs(case, seed)
        return s
    page, dim = case["page"], case["dim"]
    if case["op"] == "cache":
        s["k"], s["v"], s["slots"], n_pages = _cache_inputs(case, seed)
        heads = case["heads"]
        s["k_pages"], s["v_pages"] = (torch.zeros(n_pages, heads, _page_head_bytes(case[x], dim, page), dtype=torch.uint8, device=_device())
                                      for x in "kv")
    else:
        s.update(_attn_inputs(case, seed))
        heads = case["kv_heads"]
        s["k_pages"] = _pack(s.pop("kq"), s.pop("kd"), case["k"], "k")
        s["v_pages"] = _pack(s.pop("vq"), s.pop("vd"), case["v"], "v")
        s["max_new"] = max(_lengths(case)[1])
    for x in "kv":  # where the codes lie in a page head
        at, shift = _at(case[x], x, dim, page)
        s[x + "_at"], s[x + "_shift"] = at.to(_device()), shift.to(_device())
    if own:
        from block_quantized_matvec_amd import ft

        s["cache"] = ft.KvCache(s["k_pages"], s["v_pages"], page, heads, dim, case["k"], case["v"])
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(s):
    return {"cache": _run_cache, "attn": _run_attn, "route": _run_route}[s["case"]["op"]](s)


def _run_cache(s):
    """Writes the tokens' rows into the cache and reads the same slots back."""
    case = s["case"]
    if own:
        from block_quantized_matvec_amd import ft

        ft.kv_store(s["cache"], s["k"], s["v"], s["slots"])
        return ft.kv_load(s["cache"], s["slots"], dtype=DTYPES[case["dtype"]])
    _write(s, "k")
    _write(s, "v")
    return _read(s, "k"), _read(s, "v")


def _write(s, side):
    case, pool = s["case"], s[side + "_pages"]
    page, dim, ty, heads = case["page"], case["dim"], case[side], case["heads"]
    codes, scales = _quantize(s[side], ty)
    keep = s["slots"] >= 0
    codes, scales, slot = codes[keep], scales[keep], s["slots"][keep]
    at = s[side + "_at"][slot % page]  # [token, dim]
    base = (slot // page * heads).view(-1, 1, 1) + torch.arange(heads, device=slot.device).view(1, -1, 1)
    flat = pool.view(-1)
    where = base * pool.shape[-1] + at.unsqueeze(1)
    codes = codes.int() + (128 if ty == "Q8_0" else 8)
    if ty == "Q4_0":  # both nibbles of a byte are of one token: low and high element
        shift = s[side + "_shift"][slot % page].unsqueeze(1).expand_as(where)
        size = dim // 2
        both = torch.zeros(*where.shape[:2], size, dtype=torch.int32, device=slot.device)
        order = at.argsort(dim=1, stable=True).view(-1, 1, size, 2).expand(-1, heads, -1, -1).flatten(2)
        both = ((codes << shift.int()).gather(2, order)).unflatten(2, (size, 2)).sum(-1)
        where, codes = where.gather(2, order)[..., ::2], both
    flat[where] = codes.to(torch.uint8)
    nb = dim // 32
    held = _code_bytes(case, side)
    place = base * pool.shape[-1] + held + 2 * (torch.arange(nb, device=slot.device) * page + (slot % page).view(-1, 1)).unsqueeze(1)
    flat.view(torch.float16)[place // 2] = scales


def _code_bytes(case, side):
    return case["page"] * case["dim"] // (1 if case[side] == "Q8_0" else 2)


def _read(s, side):
    case, pool = s["case"], s[side + "_pages"]
    page, dim, ty, heads = case["page"], case["dim"], case[side], case["heads"]
    keep = s["slots"] >= 0
    slot = s["slots"].clamp(min=0)
    base = ((slot // page * heads).view(-1, 1) + torch.arange(heads, device=slot.device)).unsqueeze(-1) * pool.shape[-1]
    codes = pool.view(-1)[base + s[side + "_at"][slot % page].unsqueeze(1)].int()
    if ty == "Q4_0":
        codes = codes >> s[side + "_shift"][slot % page].unsqueeze(1).int() & 15
    codes = codes - (128 if ty == "Q8_0" else 8)
    place = base + _code_bytes(case, side) + 2 * (torch.arange(dim // 32, device=slot.device) * page + (slot % page).view(-1, 1)).unsqueeze(1)
    scales = pool.view(-1).view(torch.float16)[place // 2].float()
    x = codes.float() * scales.repeat_interleave(32, -1)
    return torch.where(keep.view(-1, 1, 1), x, torch.zeros_like(x)).to(DTYPES[case["dtype"]])


def _unpack(s, side, pages):
    """Values of whole pages: [..., pages] -> fp32 [..., kv_heads, pages * page, dim]."""
    case, pool = s["case"], s[side + "_pages"]
    page, dim, ty = case["page"], case["dim"], case[side]
    heads = pool[pages.long()]  # [..., pages, kv_heads, bytes]
    codes = heads[..., s[side + "_at"].flatten()].int()
    if ty == "Q4_0":
        codes = codes >> s[side + "_shift"].flatten().int() & 15
    codes = (codes - (128 if ty == "Q8_0" else 8)).unflatten(-1, (page, dim // 32, 32))
    scales = heads[..., _code_bytes(case, side):].contiguous().view(torch.float16).unflatten(-1, (dim // 32, page)).transpose(-1, -2)
    x = codes.float() * scales.float().unsqueeze(-1)  # [..., pages, kv_heads, page, NB, 32]
    return x.flatten(-2).movedim(-4, -3).flatten(-3, -2)


def _run_attn(s):
    case = s["case"]
    if own:
        from block_quantized_matvec_amd import ft

        return ft.attn_kv(s["cache"], s["q"], s["table"], s["kv"], s["start"], max_kv=case["kv_max"], causal=case["causal"], window=case["window"],
                          softcap=case["softcap"], slopes=s["slopes"], prefix_len=s["sinks"], n_shared=case["shared"])
    n, hk, dim, shared, new = case["n_seq"], case["kv_heads"], case["dim"], case["shared"], s["max_new"]
    group = case["heads"] // hk
    start, kv = s["start"].long(), s["kv"].long()
    # queries padded to [seq, kv_head, token * group, dim]
    count = start[1:] - start[:-1]
    step = torch.arange(new, device=kv.device)
    at = (start[:-1].view(-1, 1) + step).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(n, new, hk, group, dim).transpose(1, 2).reshape(n, hk, new * group, dim) * dim ** -0.5
    held = shared // case["page"]
    k = _unpack(s, "k", s["table"][:, held:])
    scores = torch.matmul(q, k.transpose(-1, -2))
    if shared:  # the prefix once for all: [kv_head, seq * rows, keys]
        rows = q.transpose(0, 1).reshape(hk, -1, dim)
        first = torch.matmul(rows, _unpack(s, "k", s["table"][0, :held]).transpose(-1, -2))
        scores = torch.cat([first.view(hk, n, new * group, shared).transpose(0, 1), scores], -1)
    scores = scores.view(n, hk, new, group, -1)
    pos = (kv - count).view(-1, 1) + step  # [seq, token]
    key = torch.arange(scores.shape[-1], device=kv.device)
    gap = pos.unsqueeze(-1) - key  # [seq, token, key]
    seen = torch.ones_like(gap, dtype=torch.bool)
    if case["causal"]:
        seen &= gap >= 0
    if case["window"]:
        seen &= gap < case["window"]
    if case["sinks"]:
        seen |= key < s["sinks"].view(-1, 1, 1)
    seen &= key < kv.view(-1, 1, 1)
    if case["softcap"]:
        scores = case["softcap"] * torch.tanh(scores / case["softcap"])
    if case["alibi"]:
        scores = scores - s["slopes"].view(1, hk, 1, group, 1) * gap.abs().view(n, 1, new, 1, -1)
    scores = scores.masked_fill(~seen.view(n, 1, new, 1, -1), MASKED)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - top)
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-37)).view(n, hk, new * group, -1)
    out = torch.matmul(p[..., shared:], _unpack(s, "v", s["table"][:, held:]))
    if shared:
        rows = p[..., :shared].transpose(0, 1).reshape(hk, -1, shared)
        out = out + torch.matmul(rows, _unpack(s, "v", s["table"][0, :held])).view(hk, n, new * group, dim).transpose(0, 1)
    out = out.view(n, hk, new, group, dim).transpose(1, 2).reshape(n, new, case["heads"], dim)
    return out[step < count.view(-1, 1)].to(s["q"].dtype)


def _run_route(s):
    case = s["case"]
    if own:
        from block_quantized_matvec_amd import ft

        return ft.moe_route_ex(s["logits"], case["topk"], score=case["score"], bias=s["bias"], n_group=case["groups"], topk_group=case["keep"],
                               group_top=case["top"], renorm=case["renorm"], scale=case["scale"])
    x = s["logits"].double()  # 64 bits: two experts' scores may lie next to each other
    if case["score"] == "softmax":
        score = torch.exp(x - x.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score + s["bias"].double() if case["bias"] else score
    if case["groups"] > 1:
        grouped = choice.unflatten(-1, (case["groups"], -1))
        best = grouped.sort(dim=-1, descending=True).values[..., :case["top"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[..., :case["keep"]]
        open_ = torch.zeros_like(best, dtype=torch.bool).scatter(-1, kept, True)
        choice = grouped.masked_fill(~open_.unsqueeze(-1), MASKED).flatten(-2)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[..., :case["topk"]]
    w = score.gather(-1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), (w * case["scale"]).float()


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    return {"cache": _exact_cache, "attn": _exact_attn, "route": _exact_route}[case["op"]](case, seed)


def _exact_cache(case, seed):
    k, v, slots, _ = _cache_inputs(case, seed)
    out = []
    for x, ty in ((k, case["k"]), (v, case["v"])):
        b = x.double().unflatten(-1, (-1, 32))
        if ty == "Q8_0":
            d = (b.abs().amax(-1, keepdim=True) / 127).float().half().double()
            code = (torch.floor((b / d).abs() + 0.5) * b.sign()).clamp(-127, 127)
        else:
            most, least = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
            tied = b.flatten(0, -2)[torch.arange(b.numel() // 32), b.abs().argmax(-1).flatten()].view_as(most)
            d = (torch.where(most > -least, most, torch.where(most < -least, least, tied)) / -8).float().half().double()
            code = (torch.floor((b / d).abs() + 0.5) * (b / d).sign()).clamp(-8, 7)
        y = torch.where(d == 0, torch.zeros_like(b), code * d).flatten(-2)
        y[slots < 0] = 0.0
        out.append(y)
    return tuple(out)


def _exact_attn(case, seed):
    s = _attn_inputs(case, seed)
    kv, new = _lengths(case)
    if sum(a * b for a, b in zip(kv, new)) * case["heads"] * case["dim"] > 3e11:
        return None
    group = case["heads"] // case["kv_heads"]
    outs, first = [], 0
    for i, (length, count) in enumerate(zip(kv, new)):
        q = s["q"][first:first + count].double()
        first += count
        if not length:
            outs.append(torch.zeros_like(q))
            continue
        pages = s["table"][i, :-(-length // case["page"])].long()
        pos = torch.arange(length - count, length, device=q.device).view(-1, 1)
        key = torch.arange(length, device=q.device).view(1, -1)
        seen = (key <= pos) if case["causal"] else (key >= 0).expand(count, -1)
        if case["window"]:
            seen = seen & (key > pos - case["window"])
        seen = seen | (key < case["sinks"])
        heads = []
        for h in range(case["heads"]):
            rows = []
            for codes, scales in ((s["kq"], s["kd"]), (s["vq"], s["vd"])):
                c = codes[pages, h // group].reshape(-1, case["dim"])[:length].double()
                d = scales[pages, h // group].reshape(-1, case["dim"] // 32)[:length].double()
                rows.append((c.view(length, -1, 32) * d.unsqueeze(-1)).view(length, -1))
            x = q[:, h] @ rows[0].t().contiguous() / math.sqrt(case["dim"])
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if case["alibi"]:
                x = x - s["slopes"][h].double() * (pos - key).abs()
            x = torch.softmax(x.masked_fill(~seen, MASKED), -1).nan_to_num(0.0)
            heads.append(x @ rows[1])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)


def _exact_route(case, seed):
    logits, bias = _route_inputs(case, seed)
    x = logits.double().cpu()
    score = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    choice = score + bias.double().cpu() if case["bias"] else score.clone()
    t, e, size = case["tokens"], case["experts"], case["experts"] // case["groups"]
    if case["groups"] > 1:
        best = torch.stack([torch.topk(choice[:, g * size:(g + 1) * size], min(case["top"], size)).values.sum(-1) for g in range(case["groups"])], 1)
        rank = (best.unsqueeze(1) > best.unsqueeze(2)).sum(-1)
        rank += ((best.unsqueeze(1) == best.unsqueeze(2)) & torch.ones(case["groups"], case["groups"]).tril(-1).bool()).sum(-1)
        choice[(rank >= case["keep"]).repeat_interleave(size, 1)] = MASKED
    ids = torch.empty(t, case["topk"], dtype=torch.int32)
    w = torch.empty(t, case["topk"], dtype=torch.float64)
    lowest = torch.arange(e).expand(t, -1)
    for j in range(case["topk"]):
        best = choice.amax(-1, keepdim=True)
        at = torch.where(choice == best, lowest, e).amin(-1, keepdim=True)
        ids[:, j], w[:, j] = at[:, 0].int(), score.gather(1, at)[:, 0]
        choice.scatter_(1, at, MASKED)
        choice[choice == MASKED] = MASKED
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids, w * case["scale"]
