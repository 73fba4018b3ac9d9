"""Scales that leave fp32's range in base 2 are refused (no GPU)."""
import pytest

from test_heads_cpu import INVALID, attn, lib  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scales_past_the_range(lib, scale):  # noqa: F811
    assert attn(lib, scale=scale) == INVALID


@pytest.mark.parametrize("scale", [1e-45, 1e-30, 1.0, 2.3e38])
def test_scales_within_it(lib, scale):  # noqa: F811
    assert attn(lib, scale=scale) != INVALID
