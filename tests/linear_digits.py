"""f32 operands whose three bf16 parts are known and whose partial sums are all
exact in f32, so that a lost or doubled product of parts shows."""

import numpy as np

# h in {1, 3/2} or {1, 5/4}, m = 3 2^-10, l = 3 2^-19: RN to bf16 (steps of
# 2^-7 from 1 on) of h + m + l is h, of m + l (steps of 2^-16) is m.
M, L = 3 * 2.0 ** -10, 3 * 2.0 ** -19
PAIRS = [(0, 0), (0, 1), (1, 0), (0, 2), (1, 1), (2, 0)]


def parts(rng, shape, second):
    h = rng.choice([1.0, second], size=shape)
    return np.stack([h, np.full(shape, M), np.full(shape, L)])


def product(a, b, pairs=PAIRS):
    """The sum of the products of parts, in binary64 (exact: multiples of 2^-21 below 2^20)."""
    return sum(a[i] @ b[j] for i, j in pairs)


def tolerance(terms, joined=8):
    """Relative.  The pieces of 256 terms are exact in both accumulators (multiples of 1/8 below 2^10; of 2^-21 below
    4): per piece the sum of the two and its addition to the running sum round, then up to `joined` pieces of CTAs and
    the storage; the products left out are 2 (m l) and l^2, below 2^-25."""
    return (2 * -(-terms // 256) + joined + 1) * 2.0 ** -24 + 2.0 ** -25
