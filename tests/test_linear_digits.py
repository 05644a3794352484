"""What the digits test of the f32 products can tell apart, on the CPU."""

import numpy as np
import pytest

from tests.linear_digits import L, M, PAIRS, parts, product, tolerance


def _bf16(v):
    u = np.asarray(v, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def test_the_parts_are_the_roundings():
    for second in (1.5, 1.25):
        p = parts(np.random.default_rng(0), (50,), second)
        x = p.sum(0).astype(np.float32)
        assert (x.astype(np.float64) == p.sum(0)).all()
        h = _bf16(x)
        m = _bf16(x - h)
        assert (h == p[0]).all() and (m == M).all() and (_bf16(x - h - m) == L).all()


@pytest.mark.parametrize("terms", [200, 512, 1500])
def test_a_lost_or_doubled_product_of_parts_shows(terms):
    rng = np.random.default_rng(terms)
    a, b = parts(rng, (20, terms), 1.5), parts(rng, (terms, 30), 1.25)
    want = a.sum(0) @ b.sum(0)
    off = lambda pairs: (np.abs(product(a, b, pairs) - want) / want).min()  # noqa: E731
    assert (np.abs(product(a, b) - want) / want).max() <= 2.0 ** -25
    for pair in PAIRS:
        rest = [p for p in PAIRS if p != pair]
        assert off(rest) > 2 * tolerance(terms) and off(PAIRS + [pair]) > 2 * tolerance(terms), pair
    # a part read in place of its neighbour
    for k, pair in enumerate(PAIRS):
        for other in ((pair[0], (pair[1] + 1) % 3), ((pair[0] + 1) % 3, pair[1])):
            assert off(PAIRS[:k] + [other] + PAIRS[k + 1:]) > 2 * tolerance(terms), (pair, other)
    # one operand of one part
    assert (np.abs(a[0] @ b.sum(0) - product(a, b, [(0, 0), (0, 1), (0, 2)])) == 0).all()
