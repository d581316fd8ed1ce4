"""How 4-bit attention holds a query, and that the bound its log-sums are tested with has no room for less."""
import numpy as np
import pytest

import attend4_ref as Q


@pytest.mark.parametrize("dim", [64, 128])
def test_four_numbers_leave_at_most_2_to_the_minus_19_of_the_largest(dim):
    rng = np.random.default_rng(dim)
    m = rng.integers(128, 256, (2000, dim)) * np.exp2(rng.integers(-30, 20, (2000, dim)))
    q = np.copysign(m, rng.normal(size=m.shape))  # 8 significant bits, as bf16
    left = np.abs(q - Q.held(q)).reshape(2000, -1, 32)
    top = np.abs(q).reshape(2000, -1, 32).max(-1, keepdims=True)
    assert (left <= 2.0 ** -19 * top).all()
    near = np.abs(q).reshape(2000, -1, 32) >= 2.0 ** -10 * top
    assert (left[near] == 0).all()  # all 8 bits
    assert (np.abs(q - Q.held(q, 3)).reshape(2000, -1, 32) > 2.0 ** -19 * top).any()


@pytest.mark.parametrize("dim", [64, 128])
def test_three_numbers_exceed_the_bound(dim):
    rng = np.random.default_rng(dim)
    q = Q.fine_queries(rng, 50, 1, dim)[:, 0]
    scale = dim ** -0.5
    for x in q:
        k = np.where(x > 1, 0.0, 6.0)
        bound = Q.score_bound(x, k, scale)
        assert abs(scale * ((x - Q.held(x)) @ k)) <= bound
        assert abs(scale * ((x - Q.held(x, 3)) @ k)) > 100 * bound
