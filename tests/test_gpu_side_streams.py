"""GPU: tensors that a call with `stream` makes for itself belong to that stream, as under torch.cuda.stream: the
caching allocator hands a stream's freed memory out again at once, while work on it may still be pending there."""
from types import SimpleNamespace

import pytest
import torch

from block_quantized_matvec_amd import ft, synth
from tests.gpu_util import dev, need_gpu, own_stream

pytestmark = pytest.mark.gpu

T, H, D, W = 40, 4, 64, 512


def some(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype, device="cuda")


def calls():
    cache = ft.KvCache.empty(4, 16, H, D)
    x, rows, at, slots, table = some(T, H, D), some(T, W), some(T, dtype=torch.int32), torch.arange(T, device="cuda"), some(8, D)
    ft.kv_store(cache, x, x, slots)
    ids, starts = some(T, 2, dtype=torch.int32), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    a, b, freqs = some(3, 8, W), some(3, 96, 8), some(D // 2, dtype=torch.float64)
    g = synth.rng(3)
    weights, xq = dev(synth.weights("Q4_K", 64, W, g)), ft.quantize_act("Q8_1", rows)
    bank = [dev(synth.expert_bank("Q4_K", 4, *s, g)) for s in ((256, W), (256, W), (W, 256))]
    return {
        "rope_table": lambda s: ft.rope_table(64, freqs, stream=s),
        "rope": lambda s: ft.rope(x, at, table, stream=s),
        "kv_store_rope": lambda s: ft.kv_store_rope(cache, x, x, x, slots, at, table, stream=s),
        "kv_load": lambda s: ft.kv_load(cache, slots, stream=s),
        "norm": lambda s: ft.norm(rows, residual=rows, act="Q8_1", rows=True, stream=s),
        "lora": lambda s: ft.lora(rows, a, b, at, stream=s),
        "attn_kv": lambda s: ft.attn_kv(cache, x, some(1, 3, dtype=torch.int32) * 0, starts[1:], starts, stream=s),
        "quantize_act": lambda s: ft.quantize_act("Q8_1", rows, stream=s),
        "dequant": lambda s: ft.dequant("Q4_K", weights, 64, W, stream=s),
        "mul_mat_vec_q": lambda s: ft.mul_mat_vec_q("Q4_K", weights, 64, W, "Q8_1", xq, 2, stream=s),
        "moe_route": lambda s: ft.moe_route(rows, 2, stream=s),
        "moe_route_ex": lambda s: ft.moe_route_ex(rows, 2, stream=s),
        "moe_sort": lambda s: ft.moe_sort(ids, 4, stream=s),
        "moe_q_vec": lambda s: ft.moe_q_vec("Q4_K", *bank, 4, W, 256, "Q8_K", rows[:2], ids[:2], some(2, 2), stream=s),
        "grouped_gemm_q": lambda s: ft.grouped_gemm_q("Q4_K", bank[0], 4, 256, W, "Q8_K", ft.quantize_act("Q8_K", rows), False, ids, stream=s),
    }


NAMES = ["rope_table", "rope", "kv_store_rope", "kv_load", "norm", "lora", "attn_kv", "quantize_act", "dequant", "mul_mat_vec_q", "moe_route",
         "moe_route_ex", "moe_sort", "moe_q_vec", "grouped_gemm_q"]


@pytest.mark.parametrize("name", NAMES)
def test_new_tensors_are_the_streams(name):
    need_gpu()
    f = calls()[name]
    want = f(None)
    want = [t for t in (want if isinstance(want, tuple) else (want,)) if t is not None]
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, free for the current stream's next tensors
    freed = [torch.empty_like(t) for t in want]
    places = {t.data_ptr() for t in freed}
    del freed
    stream = own_stream()
    ft.scratch_reserve(1 << 20, stream=stream)
    got = f(stream)
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() != stream
    assert not places & {t.data_ptr() for t in got}, "memory that the current stream may still use"
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_the_tables_own_angles_are_the_streams():
    """A list of angles becomes a tensor that no caller sees: it must not lie where the current stream's next tensor will."""
    need_gpu()
    freqs, _ = ft.rope_freqs(64)
    want = ft.rope_table(100, freqs)
    mine = torch.full((32,), 7.0, dtype=torch.float64, device="cuda")
    place = mine.data_ptr()
    torch.cuda.synchronize()
    del mine
    got = ft.rope_table(100, freqs, stream=own_stream())
    torch.cuda.synchronize()
    again = torch.empty(32, dtype=torch.float64, device="cuda")
    assert again.data_ptr() == place
    untouched = bool((again == 7.0).all())
    assert untouched and torch.equal(got, want)


def test_a_handle_is_enough():
    """The calls that need no device of the stream take an object with its handle alone, as ever."""
    need_gpu()
    x, stream = some(T, W), own_stream()
    torch.cuda.synchronize()
    got = ft.quantize_act("Q8_1", x, stream=SimpleNamespace(cuda_stream=stream.cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(got, ft.quantize_act("Q8_1", x))


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_stays(name):
    """Whatever the call's stream, the default one among them, and where the call is refused."""
    need_gpu()
    f, default = calls()[name], torch.cuda.default_stream()
    want = f(None)
    torch.cuda.synchronize()
    mine = own_stream()
    with torch.cuda.stream(mine):
        for stream in (default, SimpleNamespace(cuda_stream=default.cuda_stream, device=default.device), mine, None):
            got = f(stream)
            assert torch.cuda.current_stream() == mine
            torch.cuda.synchronize()
            for a, b in zip(*(t if isinstance(t, tuple) else (t,) for t in (want, got))):
                assert a is b is None or torch.equal(a, b)
        with pytest.raises((AttributeError, TypeError, ValueError)):
            f("no stream")
        assert torch.cuda.current_stream() == mine
    assert torch.cuda.current_stream() == default


def test_a_refused_call_leaves_the_stream():
    need_gpu()
    x, stream = some(T, W), own_stream()
    before = torch.cuda.current_stream()
    with pytest.raises(ft.FtError):
        ft.norm(x, act="Q8_1", eps=-1.0, stream=stream)
    with pytest.raises(ValueError):
        ft.lora(x, some(3, 8, W), some(3, 96, 8), some(T, dtype=torch.int32), out=some(T, 95), stream=stream)
    assert torch.cuda.current_stream() == before
