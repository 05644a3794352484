"""The training operators' definitions in binary64 (numpy): embedding and its
gradient, dropout, the norms' backward and the clipped policy loss, with the
bounds that a binary32 evaluation of the sums keeps."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24            # half a step of f32, relative


# ------------------------------------------------------------------ dropout

def philox4x32_10(ctr, key):
    """Philox4x32-10 (Salmon et al. 2011) of four counter words and two key
    words (integers or arrays below 2^32)."""
    mask = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in ctr]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & mask,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_keep(rows, cols, p, seed, offset):
    quads = (cols + 3) // 4
    q = np.tile(np.arange(quads, dtype=np.uint64), (rows, 1))
    r = np.tile(np.arange(rows, dtype=np.uint64)[:, None], (1, quads))
    words = philox4x32_10([q, r, offset & 0xFFFFFFFF, offset >> 32], [seed & 0xFFFFFFFF, seed >> 32])
    w = np.stack([np.broadcast_to(v, q.shape) for v in words], axis=2).reshape(rows, quads * 4)[:, :cols]
    return w >= np.uint64(round(p * 2.0 ** 32))


def dropout(x, residual, p, seed, offset):
    """f32 arrays in, the f32 result before its storage rounding (exact: one
    f32 rounding per operation)."""
    keep = dropout_keep(*x.shape, p, seed, offset)
    s = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
    with np.errstate(all="ignore"):
        y = np.where(keep, x.astype(np.float32) * s, np.float32(0))
        return y if residual is None else residual.astype(np.float32) + y


# ---------------------------------------------------------------- embedding

RUN = 32


def embed(ids, table, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    y = table[np.where(ok, ids, 0)].astype(np.float32) * np.float32(scale) if table.shape[0] else np.zeros(
        (len(ids), table.shape[1]), np.float32)
    return np.where(ok[:, None], y, np.float32(0))


def embed_backward_f32(ids, ct, vocab, scale):
    """The gradient in f32 with the declared order (runs of the sorted list);
    returns it and the mask of ids that occur."""
    ok = (ids >= 0) & (ids < vocab)
    order = np.argsort(np.where(ok, ids, vocab), kind="stable")
    out = np.zeros((vocab, ct.shape[1]), np.float32)
    seen = np.zeros(vocab, bool)
    parts = {}
    for i in range(0, int(ok.sum()), RUN):
        run = order[i:min(i + RUN, int(ok.sum()))]
        sums = {}
        for p in run:
            v = int(ids[p])
            sums[v] = sums.get(v, np.zeros(ct.shape[1], np.float32)) + ct[p].astype(np.float32)
        for v, s in sums.items():
            parts.setdefault(v, []).append(s)
    for v, ss in parts.items():
        total = ss[0]
        for s in ss[1:]:
            total = total + s
        out[v] = total * np.float32(scale)
        seen[v] = True
    return out, seen


def embed_backward(ids, ct, vocab, scale):
    """The gradient in binary64."""
    out = np.zeros((vocab, ct.shape[1]))
    ok = (ids >= 0) & (ids < vocab)
    np.add.at(out, ids[ok], ct[ok].astype(np.float64))
    return out * scale


# ------------------------------------------------------------ norm backward

def norm_backward(x, ct, gamma, kind, eps):
    """(dx, dgamma, dbeta) in binary64, each with the bound that f32 keeps: sums
    shared by at least 32 threads (ceil(n / 32) + 16 additions deep) within a
    row and taken over the rows in any order."""
    x, ct = x.astype(np.float64), ct.astype(np.float64)
    g64 = np.ones(x.shape[1]) if gamma is None else gamma.astype(np.float64)
    n = x.shape[1]
    L = (-(-n // 32) + 16) * U
    mean = lambda a: a.mean(axis=1, keepdims=True)  # noqa: E731
    g = ct * g64
    mu, mg = (mean(x), mean(g)) if kind == "layer" else (np.zeros((len(x), 1)), np.zeros((len(x), 1)))
    c = x - mu
    var = mean(c * c)
    d = np.sqrt(var + np.float64(np.float32(eps)))
    xh = c / d
    m2 = mean(g * xh)
    dx = (g - mg - xh * m2) / d
    dgamma, dbeta = (ct * xh).sum(axis=0), ct.sum(axis=0)
    # Errors: of mu, c, 1/d (relative), xh, mean g, mean(g xh), dx.
    e_mu = (L + 2 * U) * mean(np.abs(x)) if kind == "layer" else 0.0
    e_mg = (L + 3 * U) * mean(np.abs(g)) if kind == "layer" else 0.0
    e_c = e_mu + U * np.abs(c)
    e_var = (L + 3 * U) * var + 2 * mean(np.abs(c) * e_c) + mean(e_c * e_c)
    r_d = 0.5 * e_var / (d * d) + 5 * U
    e_xh = e_c / d + np.abs(xh) * (r_d + U)
    e_m2 = (L + 4 * U) * mean(np.abs(g * xh)) + mean(np.abs(g) * e_c) / d + np.abs(m2) * (r_d + 2 * U)
    e_t = U * np.abs(g) + e_mg + np.abs(m2) * e_xh + np.abs(xh) * e_m2 + e_xh * e_m2 + 3 * U * (
        np.abs(g) + np.abs(mg) + np.abs(xh * m2))
    e_dx = e_t / d + np.abs(dx) * (r_d + 2 * U)
    rows = len(x) * U
    e_dg = rows * (np.abs(ct * xh)).sum(axis=0) + (np.abs(ct) * e_xh).sum(axis=0) + U * np.abs(ct * xh).sum(axis=0)
    e_db = rows * np.abs(ct).sum(axis=0)
    tiny = 1e-36
    return (dx, e_dx + tiny), (dgamma, e_dg + tiny), (dbeta, e_db + tiny)


# -------------------------------------------------------------- policy loss

def token_logp(x, targets, scale):
    """(logp, bound, softmax, |t| = c |x - max|): logp of the targets in
    binary64 (0 for padding) and the bound of the kernels' f32 sums."""
    x = x.astype(np.float64)
    rows, cols = x.shape
    scale = np.float64(np.float32(scale))
    m = x.max(axis=1, keepdims=True)
    t = (x - m) * scale
    e = np.exp(t)
    s = e.sum(axis=1, keepdims=True)
    p = e / s
    ok = (targets >= 0) & (targets < cols)
    at = np.where(ok, targets, 0)
    logp = t[np.arange(rows), at] - np.log(s[:, 0])
    # 2^t: relative error 2^-22, of its argument 2.5 roundings; a sum at least
    # 32 threads share; the rounding of logp.
    with np.errstate(invalid="ignore"):
        et = np.where(p > 0, p * np.abs(t), 0.0).sum(axis=1)
    bound = 2.0 ** -22 + 4 * U * et + (cols / 256 + 24) * U + U * np.abs(logp)
    return np.where(ok, logp, 0.0), np.where(ok, bound, 0.0), p, np.abs(t)


def policy_loss(x, targets, old, ref, adv, weight, clip_low, clip_high, kl_coef, scale):
    """{name: (value, bound)} in binary64: loss [2], logp, dlogits."""
    rows, cols = x.shape
    ok = (targets >= 0) & (targets < cols)
    w = np.full(rows, np.float64(np.float32(1.0 / rows))) if weight is None else weight.astype(np.float64)
    live = ok & (w != 0)
    logp, e_logp = np.zeros(rows), np.zeros(rows)
    p, t = np.zeros(x.shape), np.zeros(x.shape)
    if live.any():
        logp[live], e_logp[live], p[live], t[live] = token_logp(x[live], targets[live], scale)
    a64 = adv.astype(np.float64)
    lo, hi = np.float64(np.float32(1 - clip_low)), np.float64(np.float32(1 + clip_high))
    r = np.exp(logp - old.astype(np.float64))
    bound = np.clip(r, lo, hi)
    term = -np.minimum(r * a64, bound * a64)
    d = np.where(r * a64 <= bound * a64, -a64 * r, 0.0)
    k, e1, q = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    if ref is not None:
        q = ref.astype(np.float64) - logp
        e1 = np.expm1(q)
        k = e1 - q
        d = d - kl_coef * e1
    # expf within 2 ulp, its argument's rounding; the products.
    e_r = r * (e_logp + np.abs(logp - old) * U + 6 * U)
    e_e1 = np.exp(q) * (e_logp + np.abs(q) * U) + 4 * U * np.abs(e1)
    e_term = np.abs(a64) * e_r + 2 * U * np.abs(term)
    e_k = np.abs(e1) * (e_logp + np.abs(q) * U) + 16 * U * (k + np.where(np.abs(q) >= 0.5, np.abs(e1), 0))
    e_d = np.abs(a64) * e_r + abs(kl_coef) * e_e1 + 4 * U * np.abs(d)
    out = {}
    lv = live.astype(np.float64)
    out["loss"] = (np.array([(lv * w * (term + kl_coef * k)).sum(), (lv * w * k).sum()]),
                   np.array([(lv * np.abs(w) * (e_term + abs(kl_coef) * (e_k + U * k))).sum(),
                             (lv * np.abs(w) * e_k).sum()]))
    out["loss"] = (out["loss"][0], out["loss"][1] + U * np.abs(out["loss"][0]) + 1e-36)
    out["logp"] = (logp, e_logp + 1e-36)
    sc = np.float64(np.float32(scale))
    a, e_a = lv * w * d * sc, lv * np.abs(w) * e_d * sc + 3 * U * np.abs(lv * w * d * sc)
    one = np.zeros(x.shape)
    one[np.arange(rows)[ok], targets[ok]] = 1.0
    grad = a[:, None] * (one - p)
    e_p = p * ((e_logp + 2.0 ** -22)[:, None] + 4 * U * np.where(p > 0, t, 0.0))
    # 1 - p of the target comes from logp: exp's derivative there, and 4 roundings.
    e_om = np.where(one > 0, p * e_logp[:, None] + 4 * U * np.abs(one - p), e_p)
    out["dlogits"] = (grad, e_a[:, None] * np.abs(one - p) + np.abs(a)[:, None] * (e_om + 3 * U * np.abs(one - p)) + 1e-36)
    return out
