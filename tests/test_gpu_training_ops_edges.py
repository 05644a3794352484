"""The training operators where rows begin anywhere among foreign bytes, lie
more than 2^31 elements apart, are longer than a cluster holds, and where
calls run at the same time."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.training as OT
from tests.train_util import DT, close, scratch, stored

pytestmark = pytest.mark.gpu

FAR = 1 << 22                      # elements between rows: 600 rows pass 2^31


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _amid(t, start, ld):
    """The rows of t, ld apart from element `start` of a buffer of NaN, and the buffer."""
    rows, cols = t.shape
    flat = torch.full((start + rows * ld + 16,), float("nan"), dtype=t.dtype, device=t.device)
    v = flat.as_strided((rows, cols), (ld, 1), start)
    v.copy_(t)
    return v, flat


def _untouched(flat, start, ld, rows, cols):
    keep = torch.ones(flat.shape, dtype=torch.bool, device=flat.device)
    keep.as_strided((rows, cols), (ld, 1), start).fill_(False)
    return bool(flat[keep].isnan().all())


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("rows,cols,gap", [(700, 257, 0), (333, 1001, 2), (161, 4099, 5), (3, 16383, 0), (1, 300, 0),
                                           (2, 999, 1)])
def test_norm_backward_among_foreign_bytes(R, kind, dtype, inplace, rows, cols, gap):
    rng = np.random.default_rng(rows + cols)
    x, xv = stored(rng.normal(size=(rows, cols)) + 0.25, dtype)
    c, cv = stored(rng.normal(size=(rows, cols)), dtype)
    gamma, gv = stored(1 + 0.1 * rng.normal(size=cols), "f32")
    ld = cols + gap
    x, xf = _amid(x, 3, ld)
    c, cf = _amid(c, 6, ld)
    d, df = (x, xf) if inplace else _amid(torch.zeros_like(c), 1, ld)
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = scratch(R.psk_norm_backward_workspace(rows, cols))
    eps = 1e-5
    R.psk_norm_backward(x, c, d, kind, eps, gamma, dg, db if kind == "layer" else None, ws)
    torch.cuda.synchronize()
    (wx, ex), (wg, eg), (wb, eb) = OT.norm_backward(xv, cv, gv, kind, eps)
    close(d, wx, ex, dtype)
    close(dg, wg, eg, "f32")
    if kind == "layer":
        close(db, wb, eb, "f32")
    assert _untouched(df, 3 if inplace else 1, ld, rows, cols) and _untouched(cf, 6, ld, rows, cols)
    # A sum that took a neighbour's NaN would have spread it over the row.


def _rows(rows, cols, dtype, ld):
    return torch.zeros(rows * ld, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1), 0)


def _both(call, shapes, fill):
    """call's outputs with rows close together and 2^22 elements apart, bit for bit the same.  Both lie
    on 16-byte boundaries: a row of logits is added up by the 16-byte blocks that it lies in."""
    out = []
    for far in (False, True):
        ts = {k: _rows(*s, FAR if far else (s[1] + 7) // 8 * 8) for k, s in shapes.items()}
        for k, v in fill.items():
            ts[k].copy_(v)
        extra = call(ts)
        torch.cuda.synchronize()
        out.append({k: t.contiguous().clone() for k, t in ts.items()} | extra)
        del ts
    torch.cuda.empty_cache()
    for k in out[0]:
        assert torch.equal(out[0][k], out[1][k]), k


@pytest.mark.parametrize("cols", [264, 771])
def test_rows_two_to_the_31_elements_away(R, cols):
    rows, dt = 600, torch.bfloat16
    torch.manual_seed(cols)
    a, b = (torch.randn(rows, cols, device="cuda").to(dt) for _ in range(2))
    ids = torch.randint(0, rows, (rows,), device="cuda")
    two = {"a": (rows, cols, dt), "y": (rows, cols, dt)}

    def embed(t):
        R.psk_embed(ids, t["a"], t["y"])
        return {}

    def embed_backward(t):
        R.psk_embed_backward(ids, t["a"], t["y"], workspace=scratch(R.psk_embed_workspace(rows, rows, cols)))
        return {}

    def dropout(t):
        R.psk_dropout(t["a"], t["y"], 0.25, 11)
        return {}

    def norm(t):
        dg = torch.empty(cols, device="cuda")
        R.psk_norm_backward(t["a"], t["b"], t["y"], "rms", 1e-6, None, dg, None,
                            scratch(R.psk_norm_backward_workspace(rows, cols)))
        return {"dgamma": dg}

    old, adv = torch.randn(rows, device="cuda") - 6, torch.randn(rows, device="cuda")

    def loss(t):
        out = torch.empty(2, device="cuda")
        R.psk_policy_loss(t["a"], ids % cols, old, adv, None, out, None, t["y"],
                          workspace=scratch(R.psk_policy_loss_workspace(rows, cols)))
        return {"loss": out}

    for call in (embed, embed_backward, dropout, loss):
        _both(call, two, {"a": a})
    _both(norm, two | {"b": (rows, cols, dt)}, {"a": a, "b": b})


@pytest.mark.parametrize("cols", [290001, 290008])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_beyond_a_cluster_in_place(R, cols, dtype):
    rows = 5
    torch.manual_seed(cols)
    x = torch.randn(rows, cols, device="cuda").to(DT[dtype])
    x[2].fill_(float("nan"))                     # left out: never read
    t = torch.randint(0, cols, (rows,), device="cuda")
    t[2] = -1
    old, adv = torch.randn(rows, device="cuda") - 12, torch.randn(rows, device="cuda")
    ws = scratch(R.psk_policy_loss_workspace(rows, cols))
    loss, loss2, g = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    R.psk_policy_loss(x, t, old, adv, None, loss, None, g, workspace=ws)
    R.psk_policy_loss(x, t, old, adv, None, loss2, None, x, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(x, g) and torch.equal(loss, loss2) and bool(loss.isfinite().all())
    assert not g[2].any()
    # Each live row's gradient sums to zero up to its roundings: cols terms of one sign, each within
    # half a step of its storage and 2^-20 of its size, against the one of the token.
    half = torch.finfo(DT[dtype]).eps / 2
    s, size = g.double().sum(1), g.double().abs().sum(1)
    assert bool((s.abs() <= (half + 2.0 ** -20) * size).all())


def test_calls_at_the_same_time(R):
    torch.manual_seed(5)
    rows, cols, vocab = 700, 2000, 900
    x, c = (torch.randn(rows, cols, device="cuda").to(torch.bfloat16) for _ in range(2))
    ids = torch.randint(0, vocab, (rows,), device="cuda")
    old, adv = torch.randn(rows, device="cuda") - 8, torch.randn(rows, device="cuda")

    def make():
        o = {"loss": torch.empty(2, device="cuda"), "g": torch.empty_like(x), "dx": torch.empty_like(x),
             "dg": torch.empty(cols, device="cuda"), "d": torch.empty(vocab, cols, device="cuda"),
             "wl": scratch(R.psk_policy_loss_workspace(rows, cols)),
             "wn": scratch(R.psk_norm_backward_workspace(rows, cols)),
             "we": scratch(R.psk_embed_workspace(rows, vocab, cols))}
        return [lambda: R.psk_policy_loss(x, ids, old, adv, None, o["loss"], None, o["g"], workspace=o["wl"]),
                lambda: R.psk_norm_backward(x, c, o["dx"], "rms", 1e-6, None, o["dg"], None, o["wn"]),
                lambda: R.psk_embed_backward(ids, c, o["d"], workspace=o["we"])], o

    calls, want = make()
    for f in calls:
        f()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    sets = [make() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for n, (calls, _) in enumerate(sets):
            for k, f in enumerate(calls):
                with torch.cuda.stream(streams[3 * n + k]):
                    f()
    torch.cuda.synchronize()
    for _, o in sets:
        for k in ("loss", "g", "dx", "dg", "d"):
            assert torch.equal(o[k], want[k]), k


@pytest.mark.parametrize("tokens", [300, 2000, 20000])
@pytest.mark.parametrize("cols", [264, 771])
@pytest.mark.parametrize("ids", ["few", "many", "one"])
def test_adding_to_a_leaf_is_the_leaf_plus_the_gradient(R, tokens, cols, ids):
    torch.manual_seed(tokens + cols)
    vocab = {"few": 9, "many": 1500, "one": 40}[ids]
    t = torch.full((tokens,), 17, device="cuda") if ids == "one" else torch.randint(-1, vocab, (tokens,), device="cuda")
    ct = torch.randn(tokens, cols, device="cuda").to(torch.bfloat16)
    ws = scratch(R.psk_embed_workspace(tokens, vocab, cols))
    g = torch.empty(vocab, cols, device="cuda")
    R.psk_embed_backward(t, ct, g, scale=0.75, workspace=ws)
    seen = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    seen[t[t >= 0]] = True
    assert not g[~seen].any()
    for dt in (torch.float32, torch.bfloat16):
        old = torch.randn(vocab, cols, device="cuda").to(dt)
        old[~seen] = float("nan")                # left as they are
        d = old.clone()
        R.psk_embed_backward(t, ct, d, scale=0.75, accumulate=True, workspace=ws)
        torch.cuda.synchronize()
        # One f32 rounding of the sum, one to the leaf's type.
        assert torch.equal(d[seen], (old.float() + g).to(dt)[seen])
        assert bool(d[~seen].isnan().all())
