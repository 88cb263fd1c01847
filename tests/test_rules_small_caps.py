"""Refusals of caps whose reciprocal is no float32 number: host-side checks, no
GPU needed."""

import pytest

from tests.test_rules_refusals import CALLS, _call


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("scale", [0.125, 1e-4, 0.0, -1e-4])
def test_subnormal_caps_are_refused(name, scale):
    assert _call(name, softcap=1e-40, scale=scale) == 1
    assert _call(name, softcap=5e-39, scale=scale) == 1
    assert _call(name, softcap=1.2e-38, scale=scale * 1e-3) == 0     # normal, and its product with log2(e)
