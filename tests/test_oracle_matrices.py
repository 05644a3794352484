"""The binary64 definitions of the matrix operators (oracle/matrices.py): each
gradient against central differences, and properties that pin the formulas."""

import numpy as np
import pytest

import oracle.matrices as OM


def _difference(f, x, i, h):
    a, b = x.copy(), x.copy()
    a.flat[i] += h
    b.flat[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_linear_backward_against_differences(kind):
    rng = np.random.default_rng(1)
    x, w, b, ct = rng.normal(size=(5, 4)), rng.normal(size=(4, 3)), rng.normal(size=3), rng.normal(size=(5, 3))

    def f(x, w, b):
        return (ct * OM.linear(x, w, b, kind, None, True)[0][0]).sum()

    z = x @ w + b
    (dx, _), (dw, _), (db, _) = OM.linear_backward(ct, x, w, z, kind, True, False)
    # Central differences at h = 1e-6: truncation ~ h^2, rounding ~ 1e-15 / h (no z within h of relu's corner).
    assert np.abs(z).min() > 1e-3
    for i in range(x.size):
        assert abs(_difference(lambda v: f(v, w, b), x, i, 1e-6) - dx.flat[i]) < 1e-8
    for i in range(w.size):
        assert abs(_difference(lambda v: f(x, v, b), w, i, 1e-6) - dw.flat[i]) < 1e-8
    for i in range(3):
        assert abs(_difference(lambda v: f(x, w, v), b, i, 1e-6) - db[i]) < 1e-8


@pytest.mark.parametrize("norm", ["rms", "none"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_rotary_backward_against_differences(norm, pairs):
    rng = np.random.default_rng(2)
    x, ct, gamma = rng.normal(size=(3, 2, 7)), rng.normal(size=(3, 2, 7)), rng.normal(size=7)
    ang = OM.angles([0, 5, -90001], [1.0, 0.3])
    g = gamma if norm == "rms" else None

    def f(x, gamma):
        return (ct * OM.head_norm_turn(x, ang, gamma, 1e-6, norm, pairs)[0]).sum()

    (dx, _), dg = OM.head_norm_turn_backward(ct, x, ang, g, 1e-6, norm, pairs)
    for i in range(x.size):
        assert abs(_difference(lambda v: f(v, g), x, i, 1e-6) - dx.flat[i]) < 1e-8
    if norm == "rms":
        for i in range(7):
            assert abs(_difference(lambda v: f(x, v), gamma, i, 1e-6) - dg[0][i]) < 1e-8
    else:
        assert dg is None


def test_angles_of_far_positions():
    # 2 pi as an f32 frequency: p turns, and p times what the f32 value leaves over
    f = np.float32(2 * np.pi)
    over = float(f) - 2 * np.pi
    for p in (1, 1000, 10 ** 9, -12345678):
        # 2 pi itself rounded to binary64 leaves 2.45e-16
        assert abs(OM.angles([p], [f])[0, 0] - (p * (over - 2.449e-16) + np.pi) % (2 * np.pi) + np.pi) < 1e-6


def test_turning_keeps_lengths_and_goes_back():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(4, 2, 10))
    for pairs in ("halves", "neighbours"):
        ang = OM.angles([1, 2, 3, 70000], [1.0, 0.1, 0.01])
        y = OM.turn(x, ang, pairs)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        assert np.allclose(OM.turn(y, ang, pairs, -1.0), x, rtol=0, atol=1e-12)
        assert np.array_equal(y[..., 6:], x[..., 6:])


@pytest.mark.parametrize("shape", [(6, 9), (9, 6), (7, 7)])
def test_orthogonalize_acts_on_singular_values(shape):
    rng = np.random.default_rng(4)
    g = rng.normal(size=shape)
    co = [(3.4445, -4.7750, 2.0315)] * 5
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((g * g).sum()) + 1e-7)
    for a, b, c in co:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(OM.orthogonalize(g, co, 5, 1e-7, 2.0), 2.0 * (u * s) @ v, atol=1e-9)
    near = OM.orthogonalize_rounded(g, co, 5, 1e-7, 2.0, 2) - 2.0 * (u * s) @ v
    far = OM.orthogonalize_rounded(g, co, 5, 1e-7, 2.0, 1) - 2.0 * (u * s) @ v
    assert 0 < np.abs(near).max() < 1e-4 and np.abs(near).max() < np.abs(far).max() < 0.1
