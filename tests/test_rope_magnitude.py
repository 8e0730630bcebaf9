"""The magnitude that a scaling selects (host only): a context stretched by RAMP turns heads by 0.1 ln factor + 1 times their length,
one that is not stretched by their own."""
import math

import pytest

import gated_deltanet_linear_spec_gb300 as gdn


@pytest.mark.parametrize("factor", [1e-6, math.exp(-10), math.exp(-10) * 1.0000001, 0.5, 0.999999, 1.0])
def test_ramp_of_factors_up_to_one(factor):
    """(e^-10 would make 0, which a descriptor reads as 1, and smaller ones would turn heads around.)"""
    assert gdn.Rope(64, scaling=gdn.GDN_ROPE_RAMP, factor=factor, original_len=4096, device="cpu")._desc.magnitude == 1.0


def test_a_factor_that_leaves_no_frequency_is_refused():
    with pytest.raises(gdn.GdnError, match="SHAPE"):  # 2^52 turns a position and more
        gdn.Rope(64, scaling=gdn.GDN_ROPE_RAMP, factor=1e-300, original_len=4096, device="cpu")


@pytest.mark.parametrize("factor", [1.000001, 1.5, 2.0, 40.0, 1e30])
def test_ramp_of_factors_above_one(factor):
    size = gdn.Rope(64, scaling=gdn.GDN_ROPE_RAMP, factor=factor, original_len=4096, device="cpu")._desc.magnitude
    # once in 64 bits, rounded to 32
    assert abs(size - (0.1 * math.log(factor) + 1.0)) <= 2.0 ** -23 * size and size >= 1.0


@pytest.mark.parametrize("scaling", [gdn.GDN_ROPE_PLAIN, gdn.GDN_ROPE_LINEAR, gdn.GDN_ROPE_NTK, gdn.GDN_ROPE_BANDS])
@pytest.mark.parametrize("factor", [0.25, 8.0])
def test_other_scalings_have_none(scaling, factor):
    assert gdn.Rope(64, scaling=scaling, factor=factor, original_len=4096, device="cpu")._desc.magnitude == 1.0


def test_a_given_magnitude_stays():
    assert gdn.Rope(64, scaling=gdn.GDN_ROPE_RAMP, factor=0.5, original_len=4096, magnitude=0.75, device="cpu")._desc.magnitude == 0.75
