"""The training operators' binary64 definitions (oracle/training.py): the
generator's published vectors, and each gradient against central differences
of its forward."""

import numpy as np
import pytest

import oracle.training as OT


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_published_vectors(ctr, key, want):
    assert tuple(int(v) for v in OT.philox4x32_10(ctr, key)) == want


def test_dropout_keep_rate_and_independence():
    n, p = 1 << 16, 0.3
    a, b = OT.dropout_keep(64, n // 64, p, 7, 0), OT.dropout_keep(64, n // 64, p, 7, 1)
    sigma = np.sqrt(p * (1 - p) / n)
    assert abs(a.mean() - (1 - p)) < 6 * sigma
    assert abs((a & b).mean() - (1 - p) ** 2) < 6 * sigma
    assert OT.dropout_keep(3, 5, 0.0, 1, 0).all() and not OT.dropout_keep(3, 5, 1.0, 1, 0).any()


def _difference(f, x, i, h):
    a, b = x.copy(), x.copy()
    a.flat[i] += h
    b.flat[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_backward_against_differences(kind):
    rng = np.random.default_rng(3)
    x, ct, gamma, beta = rng.normal(size=(4, 13)), rng.normal(size=(4, 13)), rng.normal(size=13), rng.normal(size=13)

    def forward(x, gamma, beta):
        c = x - x.mean(axis=1, keepdims=True) if kind == "layer" else x
        return (ct * (c / np.sqrt((c * c).mean(axis=1, keepdims=True) + np.float64(np.float32(1e-5))) * gamma
                      + beta)).sum()

    (dx, _), (dg, _), (db, _) = OT.norm_backward(x, ct, gamma, kind, 1e-5)
    # Central differences at h = 1e-5: truncation ~ h^2, rounding ~ 1e-15 / h.
    for i in range(0, x.size, 5):
        assert abs(_difference(lambda v: forward(v, gamma, beta), x, i, 1e-5) - dx.flat[i]) < 1e-8
    for i in range(13):
        assert abs(_difference(lambda v: forward(x, v, beta), gamma, i, 1e-5) - dg[i]) < 1e-8
        assert abs(_difference(lambda v: forward(x, gamma, v), beta, i, 1e-5) - db[i]) < 1e-8


def test_embedding_gradient_is_the_forwards_adjoint():
    rng = np.random.default_rng(4)
    ids, table, ct = rng.integers(-2, 9, 40), rng.normal(size=(7, 5)), rng.normal(size=(40, 5))
    grad = OT.embed_backward(ids, ct, 7, 1.5)

    def forward(t):
        ok = (ids >= 0) & (ids < 7)
        return (ct[ok] * 1.5 * t[ids[ok]]).sum()

    for i in range(table.size):
        assert abs(_difference(forward, table, i, 1e-3) - grad.flat[i]) < 1e-10
    f32, seen = OT.embed_backward_f32(ids, ct.astype(np.float32), 7, 1.5)
    assert np.abs(f32 - grad).max() < 40 * 2.0 ** -24 * 100 and list(np.nonzero(seen)[0]) == sorted(
        set(ids[(ids >= 0) & (ids < 7)]))


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_against_differences(kl):
    rng = np.random.default_rng(5)
    rows, cols = 12, 17
    x = rng.normal(size=(rows, cols)) * 2
    targets = rng.integers(0, cols, rows)
    targets[3] = -1
    logp = OT.token_logp(x, targets, 1.25)[0]
    # ratios on both sides of both bounds, away from them
    old = logp - np.log(np.resize([0.5, 0.7, 0.95, 1.1, 1.4, 2.0], rows))
    ref = logp + rng.normal(size=rows) * 0.5
    adv, w = np.resize([1.0, -1.5], rows) * rng.uniform(0.5, 2, rows), rng.uniform(0.5, 1, rows)
    adv[5:9] *= -1
    w[7] = 0.0

    def forward(v):
        return OT.policy_loss(v, targets, old, ref, adv, w, 0.2, 0.25, kl, 1.25)["loss"][0][0]

    grad = OT.policy_loss(x, targets, old, ref, adv, w, 0.2, 0.25, kl, 1.25)["dlogits"][0]
    assert not grad[3].any() and not grad[7].any()
    for i in range(0, x.size):
        assert abs(_difference(forward, x, i, 1e-6) - grad.flat[i]) < 1e-7
