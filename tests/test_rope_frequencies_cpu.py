"""Frequencies of rotary positions (host only): what is refused."""

import pytest

import w4a16_dequant_gemm_amd as W4


def test_a_ramp_needs_turns_that_differ():
    """All pairs turn alike where the base is 1 (a division by ln 1 before)."""
    with pytest.raises(ValueError):
        W4.rope_frequencies(8, 1.0, "ramp", factor=2.0, original=100, low=1.0, high=32.0, device="cpu")
    for scaling in ("none", "linear", "base", "bands"):
        freqs, m = W4.rope_frequencies(8, 1.0, scaling, factor=2.0, original=100, device="cpu")
        assert freqs.shape == (4,) and m == 1.0
