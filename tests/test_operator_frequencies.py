"""Frequencies and magnitudes at the edges of their ranges (host arithmetic, no GPU)."""

import math

import pytest

from adamw_optimizer_step_gb300 import build as build_mod
from adamw_optimizer_step_gb300 import layers


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


@pytest.mark.parametrize("factor,magnitude", [(1e-5, 1.0), (0.5, 1.0), (1.0, 1.0), (1.0 + 2.0 ** -40, 1.0),
                                              (2.0, 0.1 * math.log(2.0) + 1.0), (32.0, 0.1 * math.log(32.0) + 1.0)])
def test_yarn_magnitude(factor, magnitude):
    """0.1 ln(factor) + 1 where the context is stretched, 1 where it is not (0.1 ln 0.5 + 1 =
    0.93 would shrink queries and keys, and 0.1 ln 1e-5 + 1 is negative)."""
    spec = layers.RotarySpec(64, scaling=dict(kind="yarn", factor=factor, trained=4096.0, fast=32.0, slow=1.0))
    # the logarithm's rounding, and the float that holds the magnitude in the options
    assert abs(spec.magnitude - magnitude) <= 1e-12 and abs(spec.opts.magnitude - magnitude) <= 2.0 ** -23
