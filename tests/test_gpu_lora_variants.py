"""GPU: low-rank adapters at sizes that take the wide kernels (64 or 32 columns a wave, y and out past the L2, the coming
columns' B on its way) and the first product with four waves for 64 tokens, which smaller calls do not reach."""
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests import layer_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_lora import case, check

pytestmark = pytest.mark.gpu


def plan(t, n, many, rank):
    """(full tiles, columns a wave) that the launch takes for these sizes: csrc/ft_lora.hip's rules."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    likely = max(-(-t // 64), min(t, many))
    full = t > 64 and 16 * likely < t
    wide = likely * n >= 256 * cus and rank <= 128
    return full, likely, 16 * (1 if not wide else 2 if not full or rank > 64 else 4)


def sample(t):
    g = torch.Generator().manual_seed(t)
    rows = torch.cat([torch.arange(min(3, t)), torch.arange(max(0, t - 3), t), torch.randint(0, t, (18,), generator=g)])
    return rows.unique().cuda()


def some(out, x, a, b, ids, y, sc):
    r = sample(len(x))
    check(out[r], x[r], a, b, ids[r], y[r], sc)


def spread(ids, many, how):
    if how == "one":       # every tile of one adapter: more than 16 tokens, though the plan expects few
        ids[:] = many - 1
    elif how == "turns":   # every adapter, in turns, and none
        ids[:] = torch.arange(len(ids), dtype=torch.int32, device="cuda") % (many + 1) - 1


FULL, PART = True, False
WIDE = [(48, 14336, 32, 32, PART, 32, "any"), (48, 14339, 32, 24, PART, 32, "turns"), (40, 14345, 40, 64, PART, 32, "any"), (33, 4100, 33, 100, PART, 32, "one"),
        (512, 1411, 48, 64, PART, 32, "one"), (300, 2050, 64, 128, PART, 32, "any"), (64, 70000, 1, 16, PART, 32, "any"),
        (1500, 4097, 4, 16, FULL, 64, "any"), (1500, 4096, 3, 64, FULL, 64, "turns"), (2100, 2050, 2, 40, FULL, 64, "one"),
        (1500, 4099, 4, 100, FULL, 32, "any"), (1290, 3333, 1, 128, FULL, 32, "turns")]


@pytest.mark.parametrize("tw", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,n,many,rank,full,columns,how", WIDE)
def test_wide(t, n, many, rank, full, columns, how, tw):
    need_gpu()
    got, likely, cols = plan(t, n, many, rank)
    assert (got, cols) == (full, columns)
    x, a, b, y, ids, sc = case(t, 72, n, many, rank, "f32" if t % 2 else "bf16", tw, seed=t + rank)
    spread(ids, many, how)
    want = ft.lora(x, a, b, ids, y=y, scales=sc)
    some(want, x, a, b, ids, y, sc)
    none = (ids < 0) | (ids >= many)
    kept = torch.equal(want[none], y[none])
    assert kept
    # in place, and in rows that start anywhere
    wide = torch.full((t, n + 5), 7.0, device="cuda")
    mine = wide[:, 3:3 + n]
    mine.copy_(y)
    assert ft.lora(x, a, b, ids, y=mine, scales=sc, out=mine) is mine
    same = torch.equal(mine, want)
    assert same
    mine.fill_(7.0)
    beside = bool((wide == 7.0).all())
    assert beside
    # without y
    some(ft.lora(x, a, b, ids, scales=sc), x, a, b, ids, torch.zeros_like(y), sc)
    # a row of NaN stays in its row, and its token may be anywhere in its tile
    x[t // 2] = float("nan")
    out = ft.lora(x, a, b, ids, y=y, scales=sc)
    rest = torch.arange(t, device="cuda") != t // 2
    same = torch.equal(out[rest], want[rest])
    assert same and (bool(none[t // 2]) or bool(out[t // 2].isnan().all()))


@pytest.mark.parametrize("tx,tw", [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rank", [16, 30, 64, 200])
def test_more_tiles_than_cus(rank, tx, tw):
    """Several workgroups of 64 tokens per CU: four waves each."""
    need_gpu()
    t, k, n = 20011, 130, 90
    full, likely, _ = plan(t, n, 3, rank)
    assert full and likely > torch.cuda.get_device_properties(0).multi_processor_count
    x, a, b, y, ids, sc = case(t, k, n, 3, rank, tx, tw, seed=rank)
    out = ft.lora(x, a, b, ids, y=y, scales=sc)
    some(out, x, a, b, ids, y, sc)
    none = (ids < 0) | (ids >= 3)
    kept = torch.equal(out[none], y[none])
    assert kept


def test_long_axis_of_full_tiles():
    """Full tiles that have a CU to themselves (eight waves) and ones that share it, their long axis in shares."""
    need_gpu()
    for t, k in ((1500, 5003), (9000, 2100)):
        for tx, tw, rank in (("f32", "bf16", 64), ("bf16", "bf16", 32), ("f16", "f16", 16), ("f32", "f32", 64)):
            x, a, b, y, ids, sc = case(t, k, 300, 5, rank, tx, tw, seed=k)
            some(ft.lora(x, a, b, ids, y=y, scales=sc), x, a, b, ids, y, sc)


@pytest.mark.parametrize("t", [3, 100])
def test_pieces_cut_off(t):
    """Operands whose pieces are all as large as they can be, and of one sign: what the products of pieces leave out is
    largest, and adds up.  A value's first piece holds 8 bits, so the second is below 2^-7 of the value and the third below 2^-15;
    left out are second times third and third times second (2 * 2^-22 of the product) and third times third (2^-30).  It happens
    twice, for A x and for B h (h has what bits it has: the bound holds for any).  Sums: k and rank roundings of 2^-24 at most."""
    need_gpu()
    for tw in ("f32", "f16"):
        v = 1 + 2.0 ** -7 - 2.0 ** -23 if tw == "f32" else 1 + 2.0 ** -7 - 2.0 ** -10
        k, n, rank = 512, 40, 8
        x = torch.full((t, k), 1 + 2.0 ** -7 - 2.0 ** -23, device="cuda")
        a, b = torch.full((1, rank, k), v, device="cuda").to(ref.DT[tw]), torch.full((1, n, rank), v, device="cuda").to(ref.DT[tw])
        out = ft.lora(x, a, b, torch.zeros(t, dtype=torch.int32, device="cuda")).double()
        w = a[0, 0, 0].double().item()
        want = rank * w * (k * w * x[0, 0].double().item())
        off = ((out - want).abs() / want).max().item()
        assert off <= 2 * (2.0 ** -21 + 2.0 ** -30) + (k + rank) * 2.0 ** -24, (tw, off)
