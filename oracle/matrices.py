"""The operators of a layer's matrices in binary64 (numpy): the linear layer and
its backward, the norm and rotation of query and key heads and its backward,
the orthogonalised update -- with the bounds that the declared f32 and fp16
arithmetic keeps."""

from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24            # half a step of f32, relative
TC = 2.0 ** -23           # a tensor core's addition truncates to f32's step

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


# ------------------------------------------------------------------- linear

def act(z, kind):
    with np.errstate(all="ignore"):
        if kind == "relu":
            return np.where(z > 0, z, 0.0)
        if kind == "gelu":
            return 0.5 * z * _erfc(z * -math.sqrt(0.5))
        if kind == "silu":
            return z / (1.0 + np.exp(-z))
    return z


def act_slope(z, kind):
    with np.errstate(all="ignore"):
        if kind == "relu":
            return np.where(z > 0, 1.0, 0.0)
        if kind == "gelu":
            return 0.5 * _erfc(z * -math.sqrt(0.5)) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        if kind == "silu":
            s = 1.0 / (1.0 + np.exp(-z))
            return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


# Lipschitz bounds of the activations, and the relative error of their f32
# forms: a fit of 3.5e-7 or a reciprocal, an ex2 of 2^-22, a few roundings.
_SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1}
_ACT_ERR = {"none": 0.0, "relu": 0.0, "gelu": 16 * U, "silu": 16 * U}


def sum_error(terms, split):
    """Relative to the sum of the terms' magnitudes: the error of a tensor-core
    sum.  Each 16 products and the accumulator are added with at most 17
    truncations; with `split` operands every 256 terms go to an f32 register,
    and the products of parts left out are below 3 * 2^-24."""
    if split:
        return (17 * 16 * 2 + 4) * TC + (-(-terms // 256) + 1) * U + 4 * U
    return 17 * (-(-terms // 16) + 1) * TC


def product(a, b, split):
    """a @ b and its bound."""
    a, b = a.astype(np.float64), b.astype(np.float64)
    return a @ b, sum_error(a.shape[1], split) * (np.abs(a) @ np.abs(b)) + 1e-37


def linear(x, w, bias, kind, residual, split):
    """((y, bound), (z, bound))."""
    z, e = product(x, w, split)
    if bias is not None:
        z = z + bias
        e = e + U * (np.abs(z) + e)
    y = act(z, kind)
    ey = _SLOPE[kind] * e + _ACT_ERR[kind] * np.abs(y)
    if residual is not None:
        y = y + residual
        ey = ey + U * (np.abs(y) + ey)
    return (y, ey), (z, e)


def linear_backward(ct, x, w, z, kind, split, rounded):
    """((dx, bound), (dw, bound), (dbias, bound)); rounded: dz enters the
    products in bf16 (half a step 2^-8 ... 2^-9 relative)."""
    ct = ct.astype(np.float64)
    dz = ct if kind == "none" else ct * act_slope(z.astype(np.float64), kind)
    # the slope's absolute error: a few roundings of terms of at most 1.2
    e = np.zeros_like(dz) if kind in ("none", "relu") else np.abs(ct) * 24 * U + U * np.abs(dz)
    ep = e + 2.0 ** -8 * np.abs(dz) if rounded else e + 2.0 ** -24 * np.abs(dz)
    dx, ex = product(dz, w.T, split)
    dw, ew = product(x.T, dz, split)
    ex = ex * 1.01 + ep @ np.abs(w.T.astype(np.float64))
    ew = ew * 1.01 + np.abs(x.T.astype(np.float64)) @ ep
    rows = len(dz)
    return (dx, ex), (dw, ew), (dz.sum(0), e.sum(0) + (rows + 4) * U * np.abs(dz).sum(0) + 1e-37)


# ------------------------------------------------------------ orthogonalise

def orthogonalize(g, coefficients, steps, eps, scale):
    """The definition in binary64."""
    x = g.astype(np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    t = x.shape[0] > x.shape[1]
    x = x.T if t else x
    for i in range(steps):
        a, b, c = coefficients[i]
        q = x @ x.T
        x = a * x + (b * q + c * (q @ q)) @ x
    return scale * (x.T if t else x)


def orthogonalize_rounded(g, coefficients, steps, eps, scale, planes):
    """The same with every stored iterate rounded as the kernels hold it, all
    arithmetic in binary64: X in two fp16 parts (times 2^10), of which the
    products take `planes`; X X^T and its polynomial in `planes` parts.  Its
    distance from the definition is the size of the declared roundings."""
    def hold(v, parts):
        v = v * 1024.0
        out = np.zeros_like(v)
        for _ in range(parts):
            h = (v - out).astype(np.float16).astype(np.float64)
            out = out + h
        return out / 1024.0

    x = g.astype(np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    t = x.shape[0] > x.shape[1]
    x = hold(x.T if t else x, 2)
    for i in range(steps):
        a, b, c = coefficients[i]
        first = hold(x, planes)
        q = hold(first @ first.T, planes)
        p = hold(b * q + c * (q @ q), planes)
        x = a * x + p @ first
        if i + 1 < steps:
            x = hold(x, 2)
    return scale * (x.T if t else x)


# ------------------------------------------------------------------- rotary

def _members(dim, rot, pairs):
    j = np.arange(rot // 2)
    return (j, j + rot // 2) if pairs == "halves" else (2 * j, 2 * j + 1)


def angles(positions, freqs):
    """positions * freqs reduced to a turn (exact integers: freqs are f32), in radians."""
    out = np.empty((len(positions), len(freqs)))
    two64 = 1 << 64
    from fractions import Fraction
    inv = Fraction("0.15915494309189533576888376337251436203445964574045644874766734405889679763422654")
    for j, f in enumerate(np.asarray(freqs, dtype=np.float32)):
        turn = int(Fraction(float(f)) * inv * two64 * (1 << 40))
        for i, p in enumerate(positions):
            frac = (int(p) * turn >> 40) % two64
            frac = frac - two64 if frac >= two64 // 2 else frac
            out[i, j] = frac / two64 * 2 * math.pi
    return out


def turn(x, ang, pairs, sign=1.0):
    a, b = _members(x.shape[-1], 2 * ang.shape[1], pairs)
    c, s = np.cos(ang)[:, None, :], sign * np.sin(ang)[:, None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _turn_bound(x, e, ang, pairs):
    """The turned value's bound: cosine and sine off by 8 U (the angle's
    rounding pi U, 2 ulp of the function), two products and a sum."""
    a, b = _members(x.shape[-1], 2 * ang.shape[1], pairs)
    c, s = np.abs(np.cos(ang))[:, None, :] + 8 * U, np.abs(np.sin(ang))[:, None, :] + 8 * U
    out = e.copy()
    ma, mb = np.abs(x[..., a]), np.abs(x[..., b])
    out[..., a] = e[..., a] * c + e[..., b] * s + 12 * U * (ma + mb)
    out[..., b] = e[..., b] * c + e[..., a] * s + 12 * U * (ma + mb)
    return out


def head_norm_turn(x, ang, gamma, eps, norm, pairs):
    """(y, bound) of heads x [tokens, heads, dim]."""
    x = x.astype(np.float64)
    if norm == "rms":
        g = np.ones(x.shape[-1]) if gamma is None else gamma.astype(np.float64)
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * g
        e = (x.shape[-1] / 2 + 8) * U * np.abs(u)          # a sum of squares of dim terms (half through the root)
    else:
        u, e = x, np.zeros_like(x)
    return turn(u, ang, pairs), _turn_bound(u, e, ang, pairs) + 1e-37


def head_norm_turn_backward(ct, x, ang, gamma, eps, norm, pairs):
    """((dx, bound), (dgamma, bound))."""
    ct = ct.astype(np.float64)
    g = turn(ct, ang, pairs, -1.0)
    eg = _turn_bound(ct, np.zeros_like(ct), ang, pairs)
    if norm == "none":
        return (g, eg + 1e-37), None
    x = x.astype(np.float64)
    n = x.shape[-1]
    gam = np.ones(n) if gamma is None else gamma.astype(np.float64)
    d = np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    xh, exh = x / d, (n / 2 + 8) * U * np.abs(x / d)
    t, et = g * gam, eg * np.abs(gam) + U * np.abs(g * gam)
    m = (t * xh).mean(-1, keepdims=True)
    em = (et * np.abs(xh) + np.abs(t) * exh).mean(-1, keepdims=True) + (n + 4) * U * np.abs(t * xh).mean(-1, keepdims=True)
    dx = (t - xh * m) / d
    ed = (et + exh * np.abs(m) + np.abs(xh) * em + 3 * U * (np.abs(t) + np.abs(xh * m))) / d + (n / 2 + 8) * U * (
        np.abs(dx))
    rows = x.shape[0] * x.shape[1]
    dg = (g * xh).sum((0, 1))
    edg = (eg * np.abs(xh) + np.abs(g) * exh).sum((0, 1)) + (rows + 8) * U * np.abs(g * xh).sum((0, 1))
    return (dx, ed * 1.01 + 1e-37), (dg, edg * 1.01 + 1e-37)
