"""GPU: tensors that a call with `stream` makes for itself belong to that stream, as under torch.cuda.stream: the
caching allocator hands a stream's freed memory out again at once, while work on it may still be pending there."""
import pytest
import torch

from block_quantized_matvec_amd import ft
from tests.gpu_util import need_gpu, own_stream

pytestmark = pytest.mark.gpu


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
