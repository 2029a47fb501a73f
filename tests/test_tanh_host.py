"""The bounds of the capped scores' tanh, without a GPU: of the polynomial, and of the form beyond it with
its exponential and reciprocal rounded to nearest or a step off."""
import os
import sys

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_varlen_rotary_rope_amd", "csrc")


@pytest.fixture(scope="module")
def gen():
    sys.path.insert(0, CSRC)
    try:
        import gen_tanh_constants as m
        return m
    finally:
        sys.path.pop(0)


def test_both_forms_keep_their_bounds(gen):
    """2^-22 is promised; a step of exp2 and of the reciprocal would leave 2^-21.7, 4.93 half steps, with
    which the three other roundings of a score are still within the eight that its tests allow."""
    assert gen.worst(gen.coefficients()) < 2.0 ** -22
    assert gen.worst_far(0) < 2.0 ** -22
    for steps in (1, -1):
        assert gen.worst_far(0) < gen.worst_far(steps) < gen.MOST_BY_STEPS
    assert gen.MOST_BY_STEPS + 3 * 2.0 ** -24 < 2.0 ** -21


def test_a_nearer_border_is_noticed(gen, monkeypatch):
    """From 0.2 on the far form loses more than the bound."""
    monkeypatch.setattr(gen, "NEAR", gen.mp.mpf("0.2"))
    assert gen.worst_far(0) > 2.0 ** -22
    with pytest.raises(SystemExit):
        gen.text()
