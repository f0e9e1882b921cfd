"""The 8-bit integer oracle against its definition in exact fractions, and its products against
the dense ones."""
from fractions import Fraction

import numpy as np

from oracle import int8 as I


def _nearest(x, s):
    """Whole number nearest to x / s in exact arithmetic, ties to even."""
    f = Fraction(float(x)) / Fraction(float(s))
    lo = f.numerator // f.denominator
    rest = f - lo
    if rest != Fraction(1, 2):
        return lo + (rest > Fraction(1, 2))
    return lo + lo % 2


def test_rounding_is_that_of_exact_fractions():
    rng = np.random.default_rng(0)
    for width in (1, 7, 64):
        x = (rng.standard_normal((20, width)) * 2.0 ** rng.integers(-100, 100, (20, 1))).astype(np.float32)
        q, s = I.rows(x)
        assert np.abs(q).max() <= 127
        for r in range(20):
            for k in range(width):
                assert q[r, k] == _nearest(x[r, k], s[r])


def test_ties_go_to_even_and_the_largest_is_127():
    s = np.float32(0.75)
    x = np.concatenate([[127 * s], (np.arange(-6, 6) + 0.5) * s])[None].astype(np.float32)
    q, sc = I.rows(x)
    assert sc[0] == s and q[0, 0] == 127
    assert list(q[0, 1:]) == [-6, -4, -4, -2, -2, 0, 0, 2, 2, 4, 4, 6]


def test_zero_tiny_and_broken_rows():
    x = np.array([[0.0, 0.0], [2.0 ** -140, -2.0 ** -149], [1.0, np.inf], [np.nan, 2.0],
                  [3.4028235e38, -1e38]])
    q, s = I.rows(x)
    assert not q[:2].any() and (s[:2] == 2.0 ** -126).all()
    assert np.isnan(s[2:4]).all() and not q[2:4].any()
    assert q[4, 0] == 127 and np.isfinite(s[4])


def test_layouts_place_every_value_once():
    q = np.arange(1, 121).reshape(10, 12) % 100 + 1
    p = I.pack_weight(q)
    assert p.shape == (1, 2, 64, 16) and (p != 0).sum() == 120
    assert p[0, 0, 0, 0] == q[0, 0] and p[0, 0, 3, 9] == q[9, 3]
    tall = np.zeros((100, 17))
    tall[81, 16] = 5
    p = I.pack_weight(tall)
    assert p.shape == (2, 2, 64, 16) and p[1, 1, 16, 1] == 5 and (p != 0).sum() == 1
    assert I.pack_rows(np.ones((2, 130))).shape == (2, 256)


def test_product_and_gradient_against_the_dense_ones():
    """Within the roundings of both operands: half a scale each."""
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((9, 40)), rng.standard_normal((40, 24))
    qx, sx = I.rows(x)
    qw, sw = I.weight(w)
    got = I.product(qx, sx, qw, sw)
    bound = (0.5 * sx[:, None] * np.abs(w).sum(0) + 0.5 * sw * np.abs(I.values(qx, sx)).sum(1)[:, None])
    assert (np.abs(got - x @ w) <= bound * (1 + 1e-9)).all()
    # the gradient of sum(dc * (x @ wv)) for x, by differences (the product is linear in x)
    wv, dc = qw * sw, rng.standard_normal((9, 24))
    gate = rng.random(9)
    gq, gs = I.grad_rows(dc, np.broadcast_to(sw, dc.shape), gate)
    dx = (gq @ qw.T) * gs[:, None]
    step = 2.0 ** -10
    for r, k in ((0, 0), (3, 17), (8, 39)):
        up, dn = x.copy(), x.copy()
        up[r, k] += step
        dn[r, k] -= step
        diff = ((gate[:, None] * dc * (up @ wv)).sum() - (gate[:, None] * dc * (dn @ wv)).sum()) / (2 * step)
        assert abs(dx[r, k] - diff) <= 0.5 * gs[r] * np.abs(qw[k]).sum() + 1e-6
