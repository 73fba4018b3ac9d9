"""Head counts of the norm that 32-bit counting does not hold are refused (no GPU)."""
import pytest

from test_heads_cpu import SHAPE, heads, lib, norm  # noqa: F401  (lib is a fixture)

MOST = (1 << 31) - 256


@pytest.mark.parametrize("n", [MOST + 1, (1 << 31) - 96, (1 << 31) - 1])
def test_too_many_heads(lib, n):  # noqa: F811
    q = dict(D=8, q=heads(head=8, row=1 << 35), qo=heads(1 << 40, 1 << 35, 8))
    assert norm(lib, M=1, Hq=n, **q) == SHAPE
    assert norm(lib, M=1, Hq=1, k=heads(1 << 41, 1 << 35, 8), ko=heads(1 << 42, 1 << 35, 8), Hk=n, **q) == SHAPE


def test_most_heads_pass_the_shape_check(lib):  # noqa: F811
    assert norm(lib, M=0, Hq=MOST, D=8) != SHAPE
