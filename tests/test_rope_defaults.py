"""The angles of stretched positions where a caller leaves the turns to their defaults: those of the published methods."""
import pytest

from block_quantized_matvec_amd import ft


@pytest.mark.parametrize("scaling,high", [("blend", 4.0), ("ramp", 32.0)])
def test_default_turns(scaling, high):
    for factor, original in ((8.0, 8192), (4.0, 4096)):
        f, s = ft.rope_freqs(128, 500000.0, scaling, factor, original)
        assert (f, s) == ft.rope_freqs(128, 500000.0, scaling, factor, original, 1.0, high)
        other = ft.rope_freqs(128, 500000.0, scaling, factor, original, 1.0, 36.0 - high)
        assert f != other[0]
