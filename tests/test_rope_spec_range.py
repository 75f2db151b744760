"""Rotary specs whose parameters are in range but whose frequencies are not numbers are refused.

No GPU: the spec is a host value.  Without the refusal the fraction of a turn is
inf - floor(inf), and its conversion to an integer is undefined.
"""
import math

import pytest

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return ne.load()


@pytest.mark.parametrize("kw,word", [
    (dict(rot_dim=4, scaling="base", factor=1e-200), "base"),          # 1e4 x 1e-400: 0, and 0^(-1/2) is infinite
    (dict(rot_dim=4, scaling="base", factor=1e200), "base"),           # 1e404
    (dict(scaling="linear", factor=5e-324), "frequency"),              # 1 / 5e-324
    (dict(scaling="linear", factor=1e-308, theta=1e-300), "frequency"),
    (dict(scaling="parts", factor=5e-324, orig_len=1), "frequency"),
    (dict(mscale=1e39), "mscale"),                                     # beyond fp32, which holds it
    (dict(mscale=-1e39), "mscale"),
])
def test_specs_without_finite_angles_are_refused(kw, word):
    with pytest.raises(ne.NeError, match=word) as e:
        ne.rope_spec(64, **kw)
    assert e.value.status == ne.NE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rot_dim=4, scaling="base", factor=1e-100), dict(scaling="linear", factor=1e300),
                                dict(theta=1e300), dict(mscale=3e38), dict(mscale=0.0)])
def test_specs_at_the_far_ends_of_the_range_are_made(kw):
    """Angles per position down to 0, and an mscale that fp32 holds."""
    s = ne.rope_spec(64, **kw)
    assert math.isclose(s.mscale, kw.get("mscale", 1.0), rel_tol=2.0 ** -24)
    if "theta" in kw:
        # pair 0 turns by 1 rad whatever the base; the slowest by 1e300^(-31/32), no unit of 2^-64 of a turn
        assert abs(s.turns[0] / 2.0 ** 64 - 1 / (2 * math.pi)) <= 2.0 ** -52 and s.turns[31] == 0
