"""Cases of the matrix operators of a training step: the linear layer with its
epilogue and its gradient, the norm and rotation of queries and keys with its
gradient, and the orthogonalised update of a layer's matrices.

``own`` false: plain torch forms.  ``own`` true: the framework's entry points.
"""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
BYTES = {"bf16": 2, "f32": 4}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # a decoding step's gate product: one token for each of eight sequences
        {"name": "linear_decode", "op": "linear", "rows": 8, "cin": 2048, "cout": 5632, "dtype": "bf16",
         "act": "silu", "bias": False, "residual": False, "keep": False},
        # a training batch's first feed-forward product, z kept for the backward
        {"name": "linear_train", "op": "linear", "rows": 16384, "cin": 2048, "cout": 5632, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False, "keep": True},
        # a small f32 model of odd sizes, the branch added to the residual stream
        {"name": "linear_odd", "op": "linear", "rows": 1003, "cin": 771, "cout": 1501, "dtype": "f32",
         "act": "gelu", "bias": True, "residual": True, "keep": False},
        # the gradient of the training batch's product: activations, weights and bias
        {"name": "linear_grad_train", "op": "linear_backward", "rows": 8192, "cin": 2048, "cout": 5632,
         "dtype": "bf16", "act": "gelu"},
        # the gradient in a small f32 model of odd sizes
        {"name": "linear_grad_odd", "op": "linear_backward", "rows": 509, "cin": 771, "cout": 1003, "dtype": "f32",
         "act": "gelu"},
        # the two matrices of a small model's layer, f32
        {"name": "ortho_small", "op": "orthogonalize", "leaves": 2, "rows": 64, "cols": 192, "dtype": "f32"},
        # the query matrices of 22 layers
        {"name": "ortho_layers", "op": "orthogonalize", "leaves": 22, "rows": 2048, "cols": 2048, "dtype": "bf16"},
        # two layers' gate, up and down matrices (long side first)
        {"name": "ortho_wide", "op": "orthogonalize", "leaves": 6, "rows": 5632, "cols": 2048, "dtype": "bf16"},
        # a decoding step of eight sequences, far positions
        {"name": "rotary_decode", "op": "rotary", "rows": 8, "hq": 32, "hk": 4, "dim": 64, "rot": 64,
         "dtype": "bf16", "norm": "rms", "pairs": "halves", "far": 131072},
        # a training batch: four sequences of 4096 tokens
        {"name": "rotary_train", "op": "rotary", "rows": 16384, "hq": 32, "hk": 4, "dim": 64, "rot": 64,
         "dtype": "bf16", "norm": "rms", "pairs": "halves", "far": 0},
        # its gradient, with those of both scales
        {"name": "rotary_grad_train", "op": "rotary_backward", "rows": 16384, "hq": 32, "hk": 4, "dim": 64,
         "rot": 64, "dtype": "bf16", "norm": "rms", "pairs": "halves", "far": 0},
        # a small f32 model: heads of 50 columns of which 20 turn, neighbouring pairs
        {"name": "rotary_grad_odd", "op": "rotary_backward", "rows": 1001, "hq": 6, "hk": 6, "dim": 50, "rot": 20,
         "dtype": "f32", "norm": "rms", "pairs": "neighbours", "far": 0},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; one in two is odd or ragged."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))
    return max(lo, min(hi, n if rng.random() < 0.5 else n - n % 8 if n >= 8 else n))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "orthogonalize", "orthogonalize",
                     "rotary", "rotary", "rotary_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("linear", "linear_backward"):
        cin, cout = _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        most = (180e9 if op == "linear" else 90e9) / (cin * cout)
        rows = _spread(rng, 1, int(min(16384, most)))
        case = {"op": op, "rows": rows, "cin": cin, "cout": cout, "dtype": dtype,
                "act": rng.choice(["none", "relu", "gelu", "silu"])}
        if op == "linear":
            case |= {"bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "keep": rng.random() < 0.3}
        return case
    if op == "orthogonalize":
        rows, cols = _spread(rng, 64, 4096), _spread(rng, 64, 5632)
        short = min(rows, cols)
        cost = short * short * (3 * max(rows, cols) + short)
        leaves = rng.randint(1, max(1, min(22, int(400e9 / cost))))
        return {"op": op, "leaves": leaves, "rows": rows, "cols": cols, "dtype": dtype}
    dim = rng.choice([32, 50, 64, 80, 96, 128, 128, 256])
    hk = rng.choice([1, 2, 4, 6, 8])
    hq = hk * rng.choice([1, 2, 4, 8])
    rows = _spread(rng, 1, min(16384, 30_000_000 // ((hq + hk) * dim)))
    return {"op": op, "rows": rows, "hq": hq, "hk": hk, "dim": dim, "rot": rng.choice([dim, dim, dim // 4 * 2]),
            "dtype": dtype, "norm": rng.choice(["rms", "rms", "none"]), "pairs": rng.choice(["halves", "neighbours"]),
            "far": rng.choice([0, 0, 1000000])}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _positions(case, g):
    """Positions of sequences laid end to end; decoding steps of far sequences stand anywhere."""
    rows = case["rows"]
    if case["far"]:
        return torch.randint(0, case["far"], (rows,), generator=g, device="cuda")
    return torch.arange(rows, device="cuda") % 4096


def _update(case, g):
    """A momentum matrix: a few strong directions over noise, some rows larger than others."""
    rows, cols = case["rows"], case["cols"]
    r = max(1, min(rows, cols) // 16)
    u = _normal(g, rows, r) * torch.logspace(0, -2, r, device="cuda")
    m = u @ _normal(g, r, cols) + 0.2 * _normal(g, rows, cols)
    m = m * torch.exp(0.5 * _normal(g, rows, 1)) * 1e-3
    return m.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    if op in ("linear", "linear_backward"):
        rows, cin, cout = case["rows"], case["cin"], case["cout"]
        # normalised rows and weights of a trained layer's size
        s |= {"x": _normal(g, rows, cin, dtype=dt), "w": _normal(g, cin, cout, dtype=dt, std=cin ** -0.5)}
        if op == "linear":
            s |= {"b": _normal(g, cout, dtype=dt, std=0.1) if case["bias"] else None,
                  "res": _normal(g, rows, cout, dtype=dt) if case["residual"] else None}
        else:
            s |= {"ct": _normal(g, rows, cout, dtype=dt, std=1e-2),
                  "z": _normal(g, rows, cout, dtype=dt) if case["act"] != "none" else None}
    elif op == "orthogonalize":
        s["xs"] = [_update(case, g) for _ in range(case["leaves"])]
    else:
        rows, hq, hk, dim = case["rows"], case["hq"], case["hk"], case["dim"]
        # queries and keys are columns of the qkv product's rows
        qkv = _normal(g, rows, hq + 2 * hk, dim, dtype=dt) * 1.5
        freqs = torch.logspace(0, -math.log10(500000.0), case["rot"] // 2 + 1, device="cuda",
                               dtype=torch.float64)[:-1]
        s |= {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "pos": _positions(case, g), "freqs": freqs.float()}
        rms = case["norm"] == "rms"
        s |= {"gq": _normal(g, dim, dtype=dt, std=0.1) + 1.0 if rms else None,
              "gk": _normal(g, dim, dtype=dt, std=0.1) + 1.0 if rms else None}
        if op == "rotary_backward":
            s |= {"cq": _normal(g, rows, hq, dim, dtype=dt, std=1e-2),
                  "ck": _normal(g, rows, hk, dim, dtype=dt, std=1e-2)}
    return s


_EPS = 1e-6
_ORTHO_EPS = 1e-7
_STEPS = 5


# -------------------------------------------------------------- plain forms

def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    t = 1.0 / (1.0 + torch.exp(-z))
    return t * (1.0 + z * (1.0 - t))


def _plain_linear(s):
    dt = s["x"].dtype
    z = s["x"].float() @ s["w"].float()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(dt)}
    return out | {"z": z.to(dt)} if s["keep"] else out


def _plain_linear_backward(s):
    dt = s["x"].dtype
    dz = s["ct"].float()
    if s["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), s["act"])
    return {"dx": (dz @ s["w"].float().t()).to(dt), "dw": (s["x"].float().t() @ dz).to(dt), "dbias": dz.sum(0)}


def _plain_orthogonalize(s):
    a, b, c = COEFFICIENTS
    tall = s["rows"] > s["cols"]
    x = torch.stack([m.t() if tall else m for m in s["xs"]]).float()
    x = x / (torch.sqrt((x * x).sum((1, 2), dtype=torch.float64)).float()[:, None, None] + _ORTHO_EPS)
    for _ in range(_STEPS):
        g = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)
    return [(m.t() if tall else m).to(DTYPES[s["dtype"]]).contiguous() for m in x]


def _plain_pairs(x, s):
    """The two members of each turning pair, and the columns that do not turn."""
    rot = s["rot"]
    if s["pairs"] == "halves":
        return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]


def _plain_join(a, b, rest, s):
    turned = torch.cat([a, b], -1) if s["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_turn(x, s, sign):
    angle = s["pos"].double()[:, None, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float(), (sign * torch.sin(angle)).float()
    a, b, rest = _plain_pairs(x, s)
    return _plain_join(a * cos - b * sin, b * cos + a * sin, rest, s)


def _plain_rotary(s):
    out = {}
    for name, gamma in (("q", s["gq"]), ("k", s["gk"])):
        u = s[name].float()
        if s["norm"] == "rms":
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + _EPS) * gamma.float()
        out[name] = _plain_turn(u, s, 1.0).to(s[name].dtype)
    return out


def _plain_rotary_backward(s):
    out = {}
    for name, ct, gamma in (("q", s["cq"], s["gq"]), ("k", s["ck"], s["gk"])):
        g = _plain_turn(ct.float(), s, -1.0)
        if s["norm"] == "rms":
            x = s[name].float()
            d = torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
            xh = x / d
            t = g * gamma.float()
            out["dgamma_" + name] = (g * xh).sum((0, 1))
            g = (t - xh * (t * xh).mean(-1, keepdim=True)) / d
        out["d" + name] = g.to(s[name].dtype)
    return out


_PLAIN = {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "orthogonalize": _plain_orthogonalize,
          "rotary": _plain_rotary, "rotary_backward": _plain_rotary_backward}


# ------------------------------------------------------ the framework's calls

def _own_buffers(s, R):
    """Outputs and workspaces, made once as a training program keeps them."""
    op = s["op"]

    def new(*shape, dtype=F32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def bytes_(n):
        return torch.empty(max(16, n), device="cuda", dtype=torch.uint8)

    if op == "linear":
        shape, dt = (s["rows"], s["cout"]), s["x"].dtype
        return {"y": new(*shape, dtype=dt), "z": new(*shape, dtype=dt) if s["keep"] else None,
                "ws": bytes_(R.psk_linear_workspace(s["x"], s["w"]))}
    if op == "linear_backward":
        b = {"dx": torch.empty_like(s["x"]), "dw": torch.empty_like(s["w"]), "db": new(s["cout"])}
        return b | {"ws": bytes_(R.psk_linear_backward_workspace(s["ct"], s["x"], s["w"], b["dx"], b["dw"], b["db"],
                                                                 act=s["act"]))}
    if op == "orthogonalize":
        ys = [torch.empty_like(x) for x in s["xs"]]
        return {"ys": ys, "ws": bytes_(R.psk_orthogonalize_workspace(len(ys), s["rows"], s["cols"], ys[0].dtype))}
    b = {n: torch.empty(s[n].shape, device="cuda", dtype=s[n].dtype) for n in ("q", "k")}
    if op == "rotary_backward" and s["norm"] == "rms":
        b |= {"dgq": new(s["dim"]), "dgk": new(s["dim"]),
              "ws": bytes_(R.psk_qk_norm_rotary_backward_workspace(s["rows"], s["hq"], s["hk"], s["dim"]))}
    return b


def _run_own(s):
    import reduction_groups_gb300 as R

    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _own_buffers(s, R)
    op = s["op"]
    if op == "linear":
        R.psk_linear(s["x"], s["w"], b["y"], bias=s["b"], act=s["act"], residual=s["res"], z=b["z"],
                     workspace=b["ws"])
        return {"y": b["y"], "z": b["z"]} if s["keep"] else {"y": b["y"]}
    if op == "linear_backward":
        R.psk_linear_backward(s["ct"], s["x"], s["w"], b["dx"], b["dw"], b["db"], act=s["act"], z=s["z"],
                              workspace=b["ws"])
        return {"dx": b["dx"], "dw": b["dw"], "dbias": b["db"]}
    if op == "orthogonalize":
        R.psk_orthogonalize(s["xs"], b["ys"], steps=_STEPS, coefficients=COEFFICIENTS, eps=_ORTHO_EPS,
                            workspace=b["ws"])
        return b["ys"]
    if op == "rotary":
        R.psk_qk_norm_rotary(s["q"], s["k"], b["q"], b["k"], s["pos"], s["freqs"], s["gq"], s["gk"], norm=s["norm"],
                             eps=_EPS, pairs=s["pairs"])
        return {"q": b["q"], "k": b["k"]}
    R.psk_qk_norm_rotary_backward(s["cq"], s["ck"], s["q"], s["k"], b["q"], b["k"], s["pos"], s["freqs"], s["gq"],
                                  s["gk"], b.get("dgq"), b.get("dgk"), norm=s["norm"], eps=_EPS, pairs=s["pairs"],
                                  workspace=b.get("ws"))
    out = {"dq": b["q"], "dk": b["k"]}
    return out | {"dgamma_q": b["dgq"], "dgamma_k": b["dgk"]} if s["norm"] == "rms" else out


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("linear", "linear_backward"):
        t, k, n = case["rows"], case["cin"], case["cout"]
        if op == "linear":
            outs = 1 + case["keep"] + case["residual"]
            return {"bytes": (t * k + k * n + t * n * outs + (n if case["bias"] else 0)) * e, "flops": 2 * t * k * n}
        reads = t * k + k * n + t * n * (1 if case["act"] == "none" else 2)
        return {"bytes": (reads + t * k + k * n) * e + 4 * n, "flops": 4 * t * k * n}
    if op == "orthogonalize":
        m, n = sorted((case["rows"], case["cols"]))
        # both square products are symmetric: one triangle of each
        return {"bytes": 2 * case["leaves"] * m * n * e,
                "flops": case["leaves"] * _STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)}
    n = case["rows"] * (case["hq"] + case["hk"]) * case["dim"]
    extra = case["rows"] * 8 + 2 * case["rot"] + (2 * case["dim"] * e if case["norm"] == "rms" else 0)
    if op == "rotary":
        return {"bytes": 2 * n * e + extra, "flops": 9 * n}
    rms = case["norm"] == "rms"
    return {"bytes": (3 if rms else 2) * n * e + extra + (8 * case["dim"] if rms else 0), "flops": 16 * n}


# -------------------------------------------------------- 64-bit definitions

def _exact_act(z, kind):
    f = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu}[kind]
    return f(z)


def _exact_linear(s):
    step = max(1, 16_000_000 // s["cout"])
    w, ys, zs = s["w"].double(), [], []
    for i in range(0, s["rows"], step):
        z = torch.matmul(s["x"][i:i + step].double(), w)
        z = z if s["b"] is None else z + s["b"].double()
        y = _exact_act(z, s["act"])
        ys.append(y if s["res"] is None else y + s["res"][i:i + step].double())
        zs.append(z)
    return {"y": torch.cat(ys)} | ({"z": torch.cat(zs)} if s["keep"] else {})


def _exact_linear_backward(s):
    x = s["x"].double().requires_grad_()
    w = s["w"].double().requires_grad_()
    if s["act"] == "none":
        dz = s["ct"].double()
    else:
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(_exact_act(z, s["act"]), z, s["ct"].double())
    dx, dw = torch.autograd.grad(torch.matmul(x, w), (x, w), dz)
    return {"dx": dx, "dw": dw, "dbias": torch.matmul(torch.ones(1, len(dz), device=dz.device, dtype=dz.dtype), dz)[0]}


def _exact_orthogonalize(s):
    a, b, c = COEFFICIENTS
    out = []
    for m in s["xs"]:
        x = m.double()
        x = x / (torch.linalg.matrix_norm(x) + _ORTHO_EPS)
        for _ in range(_STEPS):
            # powers of the shorter side's product, applied from that side
            if x.shape[0] <= x.shape[1]:
                once = x @ (x.t() @ x) if x.shape[0] == x.shape[1] else (x @ x.t()) @ x
                twice = (x @ x.t()) @ once
            else:
                once = x @ (x.t() @ x)
                twice = once @ (x.t() @ x)
            x = a * x + b * once + c * twice
        out.append(x)
    return out


def _exact_rotary(s):
    """With complex numbers: a pair turns by a product with exp(i angle)."""
    leaves, out = {}, {}
    angle = s["pos"].double()[:, None, None] * s["freqs"].double()
    turn = torch.polar(torch.ones_like(angle), angle)
    rot = s["rot"]
    for name in ("q", "k"):
        x = leaves[name] = s[name].double().clone().requires_grad_()
        gamma = s["g" + name]
        u = x
        if s["norm"] == "rms":
            gamma = leaves["g" + name] = gamma.double().requires_grad_()
            u = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * gamma
        if s["pairs"] == "halves":
            v = torch.complex(u[..., :rot // 2].contiguous(), u[..., rot // 2:rot].contiguous()) * turn
            parts = [v.real, v.imag]
        else:
            v = torch.view_as_complex(u[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
            parts = [torch.view_as_real(v).flatten(-2)]
        out[name] = torch.cat(parts + [u[..., rot:]], -1)
    return leaves, out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(s)
    if op == "linear_backward":
        return _exact_linear_backward(s)
    if op == "orthogonalize":
        return _exact_orthogonalize(s)
    leaves, out = _exact_rotary(s)
    if op == "rotary":
        return {k: v.detach() for k, v in out.items()}
    res = {}
    for name in ("q", "k"):
        wanted = [leaves[name]] + ([leaves["g" + name]] if case["norm"] == "rms" else [])
        grads = torch.autograd.grad(out[name], wanted, s["c" + name].double())
        res["d" + name] = grads[0]
        if case["norm"] == "rms":
            res["dgamma_" + name] = grads[1]
    order = ["dq", "dk", "dgamma_q", "dgamma_k"] if case["norm"] == "rms" else ["dq", "dk"]
    return {k: res[k] for k in order}
