"""The cases of the linear of a few rows that lay its digits bare (CPU): a model with all eight digits is inside the bound,
one that loses any of them is not."""
import numpy as np
import pytest

import _digits_ref as D


@pytest.mark.parametrize("M,K", [(1, 512), (4, 1088), (9, 512)])
def test_every_digit_counts(M, K):
    x, w = D.make(np.random.default_rng(M + K), M, K)
    ref, tol = D.reference(x, w.double())
    off = lambda kept: (D.digits(x, kept) @ w.double().T - ref).abs() > tol  # noqa: E731
    assert not bool(off(range(8)).any())
    for lost in range(8):
        bad = off([t for t in range(8) if t != lost])
        # (digits 0 to 2 are the largest elements' and the nearest ones'; they meet weights of zero)
        assert bool(bad.any(1).all()) == (lost >= 4), lost
