"""Frequencies of rotary positions at the ends of 64 bits (no GPU needed)."""
import math

import pytest
import torch

import block_reference as ref


@pytest.fixture(scope="module")
def r():
    from w4a4_quantized_gemm_rudder_amd import rudder
    rudder.load_library()
    return rudder


@pytest.mark.parametrize("base,scaling,factor", [
    (1e-320, "plain", 1.0), (5e-324, "linear", 1e10), (5e-324, "parts", 8.0),
    (1e4, "base", 1e305), (1e300, "base", 1e10), (1e-320, "base", 1.0),
])
def test_frequencies_that_pass_64_bits_are_refused(r, base, scaling, factor):
    buf = torch.full((32,), 7.0, dtype=torch.float64)
    with pytest.raises(r.RudderError, match="passes 64 bits"):
        r.rudder_rotary_frequencies(64, base, r.ROTARY_SCALING[scaling], factor, 4096.0, 1.0, 32.0,
                                    buf)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("n,base,scaling,factor", [
    (32, 1e-300, "plain", 1.0), (32, 1e300, "plain", 1.0), (1, 5e-324, "plain", 1.0),
    (1, 1e4, "base", 1e308), (32, 1e4, "base", 1e250), (2, 1e4, "base", 1e150),
    (32, 1e300, "linear", 1e20), (16, 0.5, "parts", 4.0),
])
def test_frequencies_far_from_1(r, n, base, scaling, factor):
    got = r.rotary_frequencies(2 * n, base, scaling, factor, 4096.0, device="cpu")
    want = ref.frequencies(n, base, scaling, factor, 4096.0)
    # pow is off by some last bits of its exponent, here up to 2^10 in base 2
    assert torch.isfinite(got).all() and ((got - want).abs() <= 1e-12 * want).all()
    assert got[0] == 1 or scaling in ("linear", "parts") or math.isclose(got[0], 1)
