"""Cases of the training-step operators: the token embedding and its gradient,
dropout, the norm regions' backward and the clipped policy loss over a
vocabulary.

``own`` false: plain torch forms.  ``own`` true: the framework's entry points.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # scoring sampled answers with the current weights: one log-probability a token
        {"name": "logp_score", "op": "token_logp", "rows": 4096, "cols": 32000, "dtype": "bf16", "scale": 1.0},
        # a policy update's smallest call: a short answer, an odd vocabulary, f32 logits
        {"name": "loss_small", "op": "policy_loss", "rows": 61, "cols": 1003, "dtype": "f32", "scale": 1.0,
         "kl": 0.05, "high": 0.2, "skip": 7, "grad": True},
        # a policy update over a batch of answers sampled at temperature 1 / 1.25, prompts left out by their weight
        {"name": "loss_train", "op": "policy_loss", "rows": 8192, "cols": 32000, "dtype": "bf16", "scale": 1.25,
         "kl": 0.02, "high": 0.28, "skip": 1024, "grad": True},
        # the same over a large vocabulary, without a reference model
        {"name": "loss_wide", "op": "policy_loss", "rows": 2048, "cols": 131072, "dtype": "bf16", "scale": 1.0,
         "kl": 0.0, "high": 0.2, "skip": 100, "grad": True},
        # a decoding step's lookup: one token for each of eight sequences
        {"name": "embed_decode", "op": "embed", "rows": 8, "vocab": 32000, "cols": 2048, "dtype": "bf16", "pad": 0},
        # a training batch's lookup
        {"name": "embed_train", "op": "embed", "rows": 16384, "vocab": 32000, "cols": 2048, "dtype": "bf16",
         "pad": 300},
        # its gradient: the bf16 leaf that the optimizer reads
        {"name": "embed_grad_train", "op": "embed_backward", "rows": 16384, "vocab": 32000, "cols": 2048,
         "dtype": "bf16", "pad": 300},
        # a small batch, an odd row length, an f32 leaf
        {"name": "embed_grad_odd", "op": "embed_backward", "rows": 4099, "vocab": 5003, "cols": 771, "dtype": "f32",
         "pad": 11},
        # the dropped branch added to the residual stream
        {"name": "dropout_train", "op": "dropout", "rows": 32768, "cols": 4096, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # a small backward pass: the same mask on an f32 cotangent, odd rows
        {"name": "dropout_odd", "op": "dropout", "rows": 127, "cols": 1003, "dtype": "f32", "p": 0.5,
         "residual": False},
        # the backward of a training batch's RMSNorm, with the scale's gradient
        {"name": "norm_grad_rms", "op": "norm_backward", "rows": 32768, "cols": 4096, "dtype": "bf16", "kind": "rms"},
        # a small LayerNorm's, with scale and bias, odd rows
        {"name": "norm_grad_odd", "op": "norm_backward", "rows": 509, "cols": 771, "dtype": "f32", "kind": "layer"},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; one in two is odd or ragged."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n if rng.random() < 0.5 else n - n % 8 if n >= 8 else n))


def draw(rng):
    op = rng.choice(["token_logp", "policy_loss", "policy_loss", "embed", "embed_backward", "embed_backward",
                     "dropout", "dropout", "norm_backward", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("token_logp", "policy_loss"):
        cols = _spread(rng, 1000, 131072)
        rows = _spread(rng, 1, max(1, min(8192, 120_000_000 // cols)))
        case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "scale": rng.choice([1.0, 1.0, 0.8, 1.25])}
        if op == "policy_loss":
            case |= {"kl": rng.choice([0.0, 0.02, 0.1]), "high": rng.choice([0.2, 0.28]), "skip": rows // 9,
                     "grad": rng.random() < 0.75}
        return case
    if op in ("embed", "embed_backward"):
        cols = _spread(rng, 64, 8192)
        vocab = _spread(rng, 90, min(131072, 64_000_000 // cols))
        rows = _spread(rng, 1, min(32768, 32_000_000 // cols))
        return {"op": op, "rows": rows, "vocab": vocab, "cols": cols, "dtype": dtype, "pad": rows // 20}
    cols = _spread(rng, 64, 16384)
    rows = _spread(rng, 1, min(32768, 64_000_000 // cols))
    if op == "dropout":
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "p": rng.choice([0.05, 0.1, 0.3, 0.5]),
                "residual": rng.random() < 0.5}
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "kind": rng.choice(["rms", "layer"])}


# ------------------------------------------------------------------ inputs

def _tokens(case, g):
    """Token ids as text has them: frequencies falling with the rank as 1 / rank, ranks at random ids; `pad`
    positions hold -1."""
    rows, vocab = case["rows"], case["vocab"]
    u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).to(torch.int64).clamp_(0, vocab - 1)
    ids = torch.randperm(vocab, generator=g, device="cuda")[rank]
    ids[torch.randperm(rows, generator=g, device="cuda")[:case["pad"]]] = -1
    return ids


def _normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    rows, cols = case["rows"], case["cols"]
    s = dict(case)
    if op in ("token_logp", "policy_loss"):
        # logits with a spread of 2.5 and a sampled token between unlikely and nearly certain
        x = torch.empty(rows, cols, device="cuda", dtype=dt).normal_(0.0, 2.5, generator=g)
        t = torch.randint(0, cols, (rows,), generator=g, device="cuda")
        at = torch.arange(rows, device="cuda")
        x[at, t] += (14.0 * torch.rand(rows, generator=g, device="cuda")).to(dt)
        s |= {"logits": x, "targets": t}
        if op == "policy_loss":
            m = x.amax(1, keepdim=True).float() * case["scale"]
            lse = torch.empty(rows, device="cuda")
            step = max(1, 64_000_000 // cols)
            for i in range(0, rows, step):
                lse[i:i + step] = torch.logsumexp(x[i:i + step].float() * case["scale"] - m[i:i + step], 1)
            now = x[at, t].float() * case["scale"] - m[:, 0] - lse
            # the sampling policy is some updates behind, the reference model further
            s["old_logp"] = now + _normal(g, rows, std=0.2)
            s["ref_logp"] = now + _normal(g, rows, std=0.4) if case["kl"] else None
            s["adv"] = _normal(g, rows)
            w = torch.full((rows,), 1.0 / (rows - case["skip"]), device="cuda")
            w[torch.randperm(rows, generator=g, device="cuda")[:case["skip"]]] = 0.0
            s["weight"] = w
    elif op == "embed":
        s |= {"ids": _tokens(case, g), "table": _normal(g, case["vocab"], cols, dtype=dt, std=0.02)}
    elif op == "embed_backward":
        s |= {"ids": _tokens(case, g), "ct": _normal(g, rows, cols, dtype=dt, std=1e-2)}
    elif op == "dropout":
        s |= {"x": _normal(g, rows, cols, dtype=dt),
              "res": _normal(g, rows, cols, dtype=dt) if case["residual"] else None,
              "seed": int(torch.randint(0, 2 ** 62, (1,), generator=g, device="cuda")), "offset": 1000 + seed % 1000}
    else:
        s |= {"x": _normal(g, rows, cols, dtype=dt) + 0.25, "ct": _normal(g, rows, cols, dtype=dt, std=1e-2),
              "gamma": _normal(g, cols, dtype=dt, std=0.1) + 1.0}
    return s


def _embed_scale(case):
    return math.sqrt(case["cols"])      # rows of the table scaled to unit size, as the lookup does


_EPS = {"rms": 1e-6, "layer": 1e-5}
_CLIP_LOW = 0.2


# -------------------------------------------------------------- plain forms

def _plain_logp(s):
    """Log-probabilities of the targets in 64 bits (terms in 32), and each row's exponentials with their sum."""
    z = s["logits"].float()
    m = z.amax(1, keepdim=True)
    e = torch.exp((z - m) * s["scale"])
    total = e.sum(1, dtype=torch.float64)
    zt = z.gather(1, s["targets"][:, None])[:, 0]
    return s["scale"] * (zt.double() - m[:, 0].double()) - torch.log(total), e, total


def _plain_policy(s):
    logp, e, total = _plain_logp(s)
    w, adv = s["weight"].double(), s["adv"].double()
    r = torch.exp(logp - s["old_logp"].double())
    c = r.clamp(1.0 - _CLIP_LOW, 1.0 + s["high"])
    term = -torch.minimum(r * adv, c * adv)
    d = torch.where(r * adv <= c * adv, -adv * r, torch.zeros_like(r))
    k = torch.zeros_like(r)
    if s["kl"]:
        q = s["ref_logp"].double() - logp
        k = torch.expm1(q) - q
        d = d - s["kl"] * torch.expm1(q)
    keep = w != 0
    zero = torch.zeros_like(w)
    out = {"loss": torch.stack([torch.where(keep, w * (term + s["kl"] * k), zero).sum(),
                                torch.where(keep, w * k, zero).sum()]).float(),
           "logp": torch.where(keep, logp, zero).float()}
    if s["grad"]:
        a = (torch.where(keep, w * d, zero) * s["scale"])
        dx = e * (-a / total).float()[:, None]
        at = torch.arange(len(a), device=a.device)
        dx[at, s["targets"]] = (a - a * e[at, s["targets"]].double() / total).float()
        out["dlogits"] = torch.where(keep[:, None], dx, torch.zeros_like(dx)).to(s["logits"].dtype)
    return out


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 of 32-bit words held in int64: each wide product from two halves of its constant."""
    low = 0xFFFFFFFF

    def wide(a, m):
        hi = a * (m >> 16)
        lo = a * (m & 0xFFFF)
        t = hi + (lo >> 16)
        return t >> 16, ((t << 16) | (lo & 0xFFFF)) & low

    for _ in range(10):
        h0, l0 = wide(c0, 0xD2511F53)
        h1, l1 = wide(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _plain_dropout(s):
    rows, cols, dev = s["rows"], s["cols"], s["x"].device
    quad = torch.arange((cols + 3) // 4, device=dev).expand(rows, -1)
    row = torch.arange(rows, device=dev)[:, None].expand_as(quad)
    off = torch.full_like(quad, s["offset"])
    words = _philox(quad, row, off & 0xFFFFFFFF, off >> 32, s["seed"] & 0xFFFFFFFF, s["seed"] >> 32)
    keep = torch.stack(words, 2).reshape(rows, -1)[:, :cols] >= int(round(s["p"] * 2 ** 32))
    y = torch.where(keep, s["x"].float() * float(np.float32(1.0 / (1.0 - s["p"]))), 0.0)
    if s["res"] is not None:
        y = s["res"].float() + y
    return y.to(s["x"].dtype)


def _plain_norm_backward(s):
    x, ct = s["x"].float(), s["ct"].float()
    if s["kind"] == "layer":
        x = x - x.mean(1, keepdim=True)
    d = torch.sqrt((x * x).mean(1, keepdim=True) + _EPS[s["kind"]])
    xh = x / d
    g = ct * s["gamma"].float()
    t = g - xh * (g * xh).mean(1, keepdim=True)
    if s["kind"] == "layer":
        t = t - g.mean(1, keepdim=True)
    out = {"dx": (t / d).to(s["x"].dtype), "dgamma": (ct * xh).sum(0)}
    if s["kind"] == "layer":
        out["dbeta"] = ct.sum(0)
    return out


def _run_plain(s):
    op = s["op"]
    if op == "token_logp":
        return _plain_logp(s)[0].float()
    if op == "policy_loss":
        return _plain_policy(s)
    if op == "embed":
        ids = s["ids"]
        y = s["table"][ids.clamp(min=0)].float() * _embed_scale(s)
        return torch.where((ids >= 0)[:, None], y, torch.zeros_like(y)).to(s["table"].dtype)
    if op == "embed_backward":
        ids = s["ids"]
        ct = torch.where((ids >= 0)[:, None], s["ct"].float(), 0.0)
        d = torch.zeros(s["vocab"], s["cols"], device=ids.device).index_add_(0, ids.clamp(min=0), ct)
        return (d * _embed_scale(s)).to(s["ct"].dtype)
    if op == "dropout":
        return _plain_dropout(s)
    return _plain_norm_backward(s)


# ------------------------------------------------------ the framework's calls

def _own_buffers(s, R):
    """Outputs and workspaces, made once as a training program keeps them."""
    op, rows, cols = s["op"], s["rows"], s["cols"]

    def new(*shape, dtype=F32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def bytes_(n):
        return torch.empty(max(16, n), device="cuda", dtype=torch.uint8)

    if op == "token_logp":
        return {"logp": new(rows)}
    if op == "policy_loss":
        return {"loss": new(2), "logp": new(rows), "dlogits": torch.empty_like(s["logits"]) if s["grad"] else None,
                "ws": bytes_(R.psk_policy_loss_workspace(rows, cols))}
    if op == "embed":
        return {"y": new(rows, cols, dtype=s["table"].dtype)}
    if op == "embed_backward":
        return {"d": new(s["vocab"], cols, dtype=s["ct"].dtype),
                "ws": bytes_(R.psk_embed_workspace(rows, s["vocab"], cols))}
    if op == "dropout":
        return {"y": torch.empty_like(s["x"])}
    return {"dx": torch.empty_like(s["x"]), "dgamma": new(cols), "dbeta": new(cols) if s["kind"] == "layer" else None,
            "ws": bytes_(R.psk_norm_backward_workspace(rows, cols))}


def _run_own(s):
    import reduction_groups_gb300 as R

    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _own_buffers(s, R)
    op = s["op"]
    if op == "token_logp":
        R.psk_token_logp(s["logits"], s["targets"], b["logp"], scale=s["scale"])
        return b["logp"]
    if op == "policy_loss":
        R.psk_policy_loss(s["logits"], s["targets"], s["old_logp"], s["adv"], s["weight"], b["loss"], b["logp"],
                          b["dlogits"], ref_logp=s["ref_logp"], clip_low=_CLIP_LOW, clip_high=s["high"],
                          kl_coef=s["kl"], scale=s["scale"], workspace=b["ws"])
        out = {"loss": b["loss"], "logp": b["logp"]}
        return out | {"dlogits": b["dlogits"]} if s["grad"] else out
    if op == "embed":
        R.psk_embed(s["ids"], s["table"], b["y"], scale=_embed_scale(s))
        return b["y"]
    if op == "embed_backward":
        R.psk_embed_backward(s["ids"], s["ct"], b["d"], scale=_embed_scale(s), workspace=b["ws"])
        return b["d"]
    if op == "dropout":
        R.psk_dropout(s["x"], b["y"], s["p"], s["seed"], s["offset"], residual=s["res"])
        return b["y"]
    R.psk_norm_backward(s["x"], s["ct"], b["dx"], s["kind"], _EPS[s["kind"]], gamma=s["gamma"], dgamma=b["dgamma"],
                        dbeta=b["dbeta"], workspace=b["ws"])
    out = {"dx": b["dx"], "dgamma": b["dgamma"]}
    return out | {"dbeta": b["dbeta"]} if s["kind"] == "layer" else out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------- work

def _distinct(case):
    """Expected number of distinct ids among the non-padding positions."""
    v = np.arange(case["vocab"], dtype=np.float64)
    p = np.log1p(1.0 / (v + 1.0)) / math.log(case["vocab"] + 1)
    return float(np.sum(-np.expm1((case["rows"] - case["pad"]) * np.log1p(-p))))


def work(case):
    op, rows, cols, e = case["op"], case["rows"], case["cols"], BYTES[case["dtype"]]
    n = rows * cols
    if op == "token_logp":
        return {"bytes": n * e + rows * 12, "flops": 4 * n}
    if op == "policy_loss":
        read = (rows - case["skip"]) * cols
        return {"bytes": (read + (n if case["grad"] else 0)) * e + rows * (28 if case["kl"] else 24),
                "flops": (8 if case["grad"] else 4) * read}
    if op == "embed":
        return {"bytes": rows * 8 + (_distinct(case) * cols + n) * e, "flops": n}
    if op == "embed_backward":
        return {"bytes": rows * 8 + (rows - case["pad"] + case["vocab"]) * cols * e, "flops": n}
    if op == "dropout":
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": 2 * n}
    return {"bytes": 3 * n * e + cols * (e + (8 if case["kind"] == "layer" else 4)), "flops": 14 * n}


# -------------------------------------------------------- 64-bit definitions

def _exact_loss(s):
    rows, cols = s["rows"], s["cols"]
    step = max(1, 32_000_000 // cols)
    logp, grads = [], []
    at = [slice(i, min(rows, i + step)) for i in range(0, rows, step)]
    for a in at:
        lp = torch.log_softmax(s["logits"][a].double() * s["scale"], 1)
        logp.append(lp.gather(1, s["targets"][a, None])[:, 0])
    logp = torch.cat(logp)
    if s["op"] == "token_logp":
        return logp
    live = s["weight"] != 0
    leaf = logp.clone().requires_grad_()
    ratio = (leaf - s["old_logp"].double()).exp()
    adv = s["adv"].double()
    low, high = 1 - _CLIP_LOW, 1 + s["high"]
    bounded = torch.where(ratio < low, low, torch.where(ratio > high, high, ratio))
    term = torch.where(ratio * adv > bounded * adv, -bounded * adv, -ratio * adv)
    k = torch.zeros_like(term)
    if s["kl"]:
        q = s["ref_logp"].double() - leaf
        k = q.expm1() - q
    w = s["weight"].double()
    loss = (w * (term + s["kl"] * k))[live].sum()
    out = {"loss": torch.stack([loss.detach(), (w * k)[live].sum().detach()]), "logp": torch.where(live, logp, 0.0)}
    if s["grad"]:
        loss.backward()
        c = leaf.grad * s["scale"]
        for a in at:
            d = torch.softmax(s["logits"][a].double() * s["scale"], 1).neg_()
            d.scatter_add_(1, s["targets"][a, None], torch.ones_like(d[:, :1]))
            grads.append(torch.where(live[a, None], d * c[a, None], 0.0))
        out["dlogits"] = torch.cat(grads)
    return out


def _exact_keep(s, first, rows):
    """The kept positions of `rows` rows from row `first`: Philox4x32-10 in numpy's 64-bit unsigned words."""
    cols = s["cols"]
    nq = (cols + 3) // 4
    u, mask = np.uint64, np.uint64(0xFFFFFFFF)
    x = [np.tile(np.arange(nq, dtype=u), rows), np.repeat(np.arange(first, first + rows, dtype=u), nq),
         u(s["offset"] & 0xFFFFFFFF), u(s["offset"] >> 32)]
    key = [s["seed"] & 0xFFFFFFFF, s["seed"] >> 32]
    for r in range(10):
        a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        ka, kb = ((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), ((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        x = [(b >> u(32)) ^ x[1] ^ u(ka), b & mask, (a >> u(32)) ^ x[3] ^ u(kb), a & mask]
    words = np.stack([np.broadcast_to(w, (rows * nq,)) for w in x], 1).reshape(rows, nq * 4)[:, :cols]
    return words >= u(int(round(s["p"] * 2.0 ** 32)))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("token_logp", "policy_loss"):
        return _exact_loss(s)
    if op == "embed":
        t = torch.nn.functional.pad(s["table"].double() * _embed_scale(case), (0, 0, 0, 1))
        return t[torch.where(s["ids"] < 0, case["vocab"], s["ids"])]
    if op == "embed_backward":
        ids = s["ids"].cpu().numpy()
        order = np.argsort(ids, kind="stable")[np.count_nonzero(ids < 0):]
        out = np.zeros((case["vocab"], case["cols"]))
        if order.size:
            v, start = np.unique(ids[order], return_index=True)
            out[v] = np.add.reduceat(s["ct"].double().cpu().numpy()[order], start, axis=0) * _embed_scale(case)
        return torch.from_numpy(out)
    if op == "dropout":
        rows, step = case["rows"], max(1, 1_000_000 // case["cols"])
        keep = np.concatenate([_exact_keep(s, i, min(step, rows - i)) for i in range(0, rows, step)])
        keep = torch.from_numpy(keep).to(s["x"].device)
        y = s["x"].double() / (1.0 - case["p"]) * keep
        return y if s["res"] is None else y + s["res"].double()
    x = s["x"].double().requires_grad_()
    gamma = s["gamma"].double().requires_grad_()
    beta = torch.zeros_like(gamma).requires_grad_()
    if case["kind"] == "layer":
        y = torch.nn.functional.layer_norm(x, (case["cols"],), gamma, beta, _EPS["layer"])
    else:
        y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + _EPS["rms"]) * gamma
    y.backward(s["ct"].double())
    out = {"dx": x.grad, "dgamma": gamma.grad}
    return out | {"dbeta": beta.grad} if case["kind"] == "layer" else out
