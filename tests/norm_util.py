"""How far whole output vectors may be off: the elementwise parity bound adds absolute sums through
two chained products and lets an error of 1e-4 of the result pass."""

import numpy as np

# A product in 32 bits moves its output vector by at most (K / 256 + 8) 2^-24 of itself for the sums
# of K <= 1024 elements (7e-7, all roundings one way), 4 2^-23 for the matrix unit's truncated sums
# of a block (5e-7) and, where x is held in two f16 parts, 2^-22 (2.4e-7).  Gate and up (together at
# most 1.1 + 1 times that) and down follow one another: 3.1 * 1.4e-6 at the very most, and about a
# fifth of it with roundings of either sign.  Plain f16 in place of the two parts: 3e-4.
NORM_TOL = 3e-6


def norm_error(got, want):
    """Largest ||got - want|| / ||want|| over the rows."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    return float(np.max(np.linalg.norm(got - want, axis=-1) / np.linalg.norm(want, axis=-1)))


def assert_norms(got, want, what="", tol=NORM_TOL):
    e = norm_error(got, want)
    assert e <= tol, "%s: an output vector is off by %.3g of itself (at most %.3g)" % (what, e, tol)
    return e
