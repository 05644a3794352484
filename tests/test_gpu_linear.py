"""psk_linear and psk_linear_backward against their binary64 definition, within
the bounds of the declared sums and storage roundings."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.guard import guarded
from tests.train_util import DT, close, scratch, stored, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _weight(rng, cin, cout, wt, layout, pad):
    v = rng.normal(size=(cin, cout)) / max(1, cin) ** 0.5
    w, wv = stored(v if layout == "in_out" else v.T, wt)
    w = strided(w, *pad) if pad else w
    return (w, wv) if layout == "in_out" else (w.t(), wv.T)


def _forward(R, rows, cin, cout, xt="bf16", wt=None, yt=None, zt=None, act="none", bias=None, res=None, layout="in_out",
             pad=None, inplace=False, seed=0):
    rng = np.random.default_rng(rows * 7 + cin * 3 + cout + seed)
    wt, yt = wt or xt, yt or xt
    x, xv = stored(rng.normal(size=(rows, cin)), xt)
    x = strided(x, *pad) if pad else x
    w, wv = _weight(rng, cin, cout, wt, layout, pad)
    b, bv = stored(rng.normal(size=cout), bias) if bias else (None, None)
    r, rv = stored(rng.normal(size=(rows, cout)), res) if res else (None, None)
    gy, gz = guarded((rows, cout), DT[yt]), guarded((rows, cout), DT[zt or "f32"])
    y = gy.tensor
    if pad:
        y = strided(y, *pad)
        r = strided(r, *pad) if res else None
    if inplace:
        y = r
    R.psk_linear(x, w, y, b, act, r, gz.tensor if zt else None, workspace=scratch(R.psk_linear_workspace(x, w)))
    torch.cuda.synchronize()
    assert gy.intact() and gz.intact()
    (wy, ey), (wz, ez) = OM.linear(xv, wv, bv, act, rv, "f32" in (xt, wt))
    close(y, wy, ey, yt)
    if zt:
        close(gz.tensor, wz, ez, zt)
    else:
        assert bool(gz.tensor.isnan().all())


SHAPES = [(1, 1, 1), (1, 64, 8), (3, 5, 7), (8, 2048, 256), (128, 64, 128), (129, 65, 257), (77, 771, 1003),
          (300, 256, 512), (500, 100, 30), (256, 1024, 768), (2, 4096, 40), (33, 63, 1), (1000, 8, 24), (17, 640, 4104)]


@pytest.mark.parametrize("rows,cin,cout", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_against_binary64(R, rows, cin, cout, dtype, layout):
    _forward(R, rows, cin, cout, dtype, layout=layout)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("rows,cin,cout,dtype", [(300, 192, 264, "bf16"), (77, 101, 131, "bf16"), (70, 96, 200, "f32"),
                                                 (4, 512, 1030, "bf16")])
def test_epilogue(R, act, rows, cin, cout, dtype):
    other = {"bf16": "f32", "f32": "bf16"}[dtype]
    _forward(R, rows, cin, cout, dtype, act=act, bias=dtype, res=dtype, zt=dtype)
    _forward(R, rows, cin, cout, dtype, act=act, bias=other, res=other, zt=other, yt=other)
    _forward(R, rows, cin, cout, dtype, act=act, res=dtype, inplace=True)


@pytest.mark.parametrize("xt,wt,yt", [("bf16", "f32", "bf16"), ("f32", "bf16", "f32"), ("bf16", "bf16", "f32"),
                                      ("f32", "f32", "bf16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("rows,cin,cout", [(130, 200, 136), (9, 33, 50)])
def test_mixed_types(R, xt, wt, yt, rows, cin, cout):
    _forward(R, rows, cin, cout, xt, wt, yt, bias="f32", act="silu")


@pytest.mark.parametrize("pad", [(8, 0), (8, 8), (3, 1), (5, 0), (8, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_strided(R, pad, dtype, layout):
    _forward(R, 140, 200, 264, dtype, act="gelu", bias=dtype, res=dtype, layout=layout, pad=pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cin,cout", [(2000, 1024, 1536), (1024, 2048, 2056), (700, 3000, 520), (64, 8192, 300)])
def test_many_tiles(R, rows, cin, cout, dtype):
    _forward(R, rows, cin, cout, dtype, act="gelu", bias=dtype, zt=dtype)


def test_f32_operands_keep_their_digits(R):
    """One term a sum: the product to f32, whatever the split of the operands drops (three products below 2^-24
    together, three truncations, the accumulator's order)."""
    rng = np.random.default_rng(5)
    scale = 10.0 ** rng.uniform(-15, 15, size=(200, 1))
    x, xv = stored(rng.normal(size=(200, 1)) * scale, "f32")
    w, wv = stored(rng.normal(size=(1, 100)), "f32")
    y = torch.empty(200, 100, device="cuda")
    R.psk_linear(x, w, y, workspace=scratch(R.psk_linear_workspace(x, w)))
    want = xv.astype(np.float64) * wv.astype(np.float64)
    assert (np.abs(y.cpu().numpy() - want) <= 12 * 2.0 ** -24 * np.abs(want)).all()


def test_gelu_keeps_its_tail(R):
    z = torch.linspace(-13.5, 13.5, 2001, device="cuda")[:, None].contiguous()
    one = torch.ones(1, 1, device="cuda")
    for act in ("gelu", "silu"):
        y = torch.empty_like(z)
        R.psk_linear(z, one, y, act=act, workspace=scratch(R.psk_linear_workspace(z, one)))
        zv = z.cpu().numpy().astype(np.float64)
        want = OM.act(zv, act)
        # z off by three truncations: |z^2| of them in the tail's exponent; the function's 16 U
        bound = (16 + 8 * (1 + zv * zv)) * 2.0 ** -24 * np.abs(want) + 1e-37
        assert (np.abs(y.cpu().numpy() - want) <= bound).all(), act


def test_infinite_and_nan_rows_stay_in_their_rows(R):
    rng = np.random.default_rng(6)
    for dtype in ("bf16", "f32"):
        x, _ = stored(rng.normal(size=(40, 70)), dtype)
        w, _ = stored(rng.normal(size=(70, 50)), dtype)
        x[3, 5], x[9, 0], w[7, 11] = float("nan"), float("inf"), float("nan")
        y = torch.empty(40, 50, device="cuda", dtype=DT[dtype])
        R.psk_linear(x, w, y, act="gelu", workspace=scratch(R.psk_linear_workspace(x, w)))
        ok = y.isfinite()
        assert bool(y[3].isnan().all()) and bool(y[:, 11].isnan().all())
        ok[3], ok[9], ok[:, 11] = True, True, True
        assert bool(ok.all())
    b = torch.tensor([float("inf"), float("-inf"), 1.0], device="cuda")
    x, w, y = torch.ones(2, 1, device="cuda"), torch.zeros(1, 3, device="cuda"), torch.empty(2, 3, device="cuda")
    for act in ("relu", "gelu", "silu"):
        R.psk_linear(x, w, y, b, act, workspace=scratch(R.psk_linear_workspace(x, w)))
        assert bool(y[:, 0].isposinf().all()) and bool((y[:, 1] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_to_sum(R, dtype):
    x, w = torch.empty(5, 0, device="cuda", dtype=DT[dtype]), torch.empty(0, 9, device="cuda", dtype=DT[dtype])
    b, y = torch.arange(9, device="cuda", dtype=DT[dtype]), torch.full((5, 9), float("nan"), device="cuda")
    R.psk_linear(x, w, y, b, "relu", workspace=scratch(R.psk_linear_workspace(x, w)))
    assert torch.equal(y, b.float().expand(5, 9))
    R.psk_linear(torch.empty(0, 4, device="cuda"), torch.empty(4, 9, device="cuda"), y[:0])
    R.psk_linear(torch.empty(3, 4, device="cuda"), torch.empty(4, 0, device="cuda"), y[:3, :0])


def _backward(R, rows, cin, cout, dtype="bf16", act="none", layout="in_out", accumulate=False, outs=None, pad=None,
              want="xwb", dbt="f32", types=None, seed=0):
    rng = np.random.default_rng(rows * 5 + cin + cout * 3 + seed)
    xt, wt, ct_t = types or (dtype, dtype, dtype)
    dxt, dwt = outs or (xt, wt)
    x, xv = stored(rng.normal(size=(rows, cin)), xt)
    ct, cv = stored(rng.normal(size=(rows, cout)), ct_t)
    z, zv = stored(rng.normal(size=(rows, cout)), dtype)
    x, ct, z = (strided(t, *pad) for t in (x, ct, z)) if pad else (x, ct, z)
    w, wv = _weight(rng, cin, cout, wt, layout, pad)
    gx, gb = guarded((rows, cin), DT[dxt]), guarded((cout,), DT[dbt])
    gw = guarded((cin, cout) if layout == "in_out" else (cout, cin), DT[dwt])
    dw0, dw0v = stored(rng.normal(size=tuple(gw.tensor.shape)), dwt)
    db0, db0v = stored(rng.normal(size=cout), dbt)
    if accumulate:
        gw.tensor.copy_(dw0)
        gb.tensor.copy_(db0)
    dw = gw.tensor if layout == "in_out" else gw.tensor.t()
    dx, dw, db = (t if k in want else None for k, t in zip("xwb", (gx.tensor, dw, gb.tensor)))
    ws = scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw, db, act=act))
    R.psk_linear_backward(ct, x, w, dx, dw, db, act=act, z=None if act == "none" else z, accumulate=accumulate,
                          workspace=ws)
    torch.cuda.synchronize()
    assert gx.intact() and gw.intact() and gb.intact()
    for name, kind, got, dt, first in (("x", 0, dx, dxt, None), ("w", 1, dw, dwt, dw0v), ("b", 2, db, dbt, db0v)):
        if got is None:
            continue
        other, own = (wt, dxt) if name == "x" else (xt, dwt)
        split = "f32" in (ct_t, other) or (act != "none" and own == "f32")
        rounded = act != "none" and not split
        wantv, bound = OM.linear_backward(cv, xv, wv, zv, act, split, rounded)[kind]
        if accumulate and first is not None:
            f = first.astype(np.float64)
            wantv = wantv + (f if name == "b" or layout == "in_out" else f.T)
            bound = bound + 2.0 ** -24 * np.abs(wantv)
        close(got, wantv, bound, dt)
    for k, g in zip("xwb", (gx, gw, gb)):
        if k not in want and not accumulate:
            assert bool(g.tensor.isnan().all())


@pytest.mark.parametrize("rows,cin,cout", [(1, 1, 1), (3, 5, 7), (128, 64, 128), (77, 771, 503), (300, 200, 104),
                                           (1000, 64, 40), (257, 129, 600), (40, 1000, 8)])
@pytest.mark.parametrize("dtype,act", [("bf16", "none"), ("bf16", "gelu"), ("f32", "none"), ("f32", "silu"),
                                       ("bf16", "relu")])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_backward_against_binary64(R, rows, cin, cout, dtype, act, layout):
    _backward(R, rows, cin, cout, dtype, act, layout)


@pytest.mark.parametrize("dtype,act", [("bf16", "none"), ("bf16", "silu"), ("f32", "gelu")])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_backward_adds_to_the_leaf(R, dtype, act, layout):
    _backward(R, 130, 96, 72, dtype, act, layout, accumulate=True)
    _backward(R, 65, 33, 51, dtype, act, layout, accumulate=True, dbt="bf16")


@pytest.mark.parametrize("want", ["x", "w", "b", "xw", "xb", "wb"])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_unwanted_gradients(R, want, act):
    _backward(R, 70, 88, 104, "bf16", act, want=want)
    _backward(R, 70, 33, 21, "f32", act, want=want)


@pytest.mark.parametrize("types,outs", [(("bf16", "bf16", "bf16"), ("f32", "f32")), (("bf16", "bf16", "bf16"), ("bf16", "f32")),
                                        (("bf16", "bf16", "f32"), ("bf16", "bf16")), (("f32", "bf16", "bf16"), ("bf16", "f32")),
                                        (("bf16", "f32", "bf16"), ("bf16", "f32"))])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_mixed_types(R, types, outs, act):
    _backward(R, 200, 72, 136, "bf16", act, types=types, outs=outs)


@pytest.mark.parametrize("pad", [(8, 0), (3, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_strided(R, pad, dtype):
    _backward(R, 140, 200, 264, dtype, "gelu", pad=pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_many_tiles(R, dtype):
    _backward(R, 2048, 1024, 1536, dtype, "gelu")
    _backward(R, 3000, 520, 300, dtype, "none")


def test_backward_of_no_rows(R):
    e = lambda *s: torch.full(s, 3.0, device="cuda")  # noqa: E731
    x, w, ct = e(0, 16), e(16, 8), e(0, 8)
    for acc, left in ((False, 0.0), (True, 3.0)):
        dw, db = e(16, 8), e(8)
        ws = scratch(R.psk_linear_backward_workspace(ct, x, w, None, dw, db, act="gelu"))
        R.psk_linear_backward(ct, x, w, None, dw, db, act="gelu", z=ct, accumulate=acc, workspace=ws)
        assert bool((dw == left).all()) and bool((db == left).all())


def test_slopes_at_the_ends(R):
    z = torch.tensor([[float("inf"), float("-inf"), 0.0, 40.0, -40.0, -200.0]], device="cuda")
    ct, db = torch.ones(1, 6, device="cuda"), torch.empty(6, device="cuda")
    x, w = torch.empty(1, 1, device="cuda"), torch.empty(1, 6, device="cuda")
    for act, want in (("relu", [1, 0, 0, 1, 0, 0]), ("gelu", [1, 0, 0.5, 1, 0, 0]), ("silu", [1, 0, 0.5, 1, 0, 0])):
        R.psk_linear_backward(ct, x, w, None, None, db, act=act, z=z,
                              workspace=scratch(R.psk_linear_backward_workspace(ct, x, w, None, None, db, act=act)))
        # silu'(-40) = -39 exp(-40)
        assert torch.allclose(db, torch.tensor(want, device="cuda", dtype=torch.float32), rtol=0, atol=1e-15), act


def test_gradients_against_differences_of_the_forward(R):
    """The directional derivative of sum(ct y), from the library's own forward in f32 with steps of 2^-6."""
    rng = np.random.default_rng(8)
    x, _ = stored(rng.normal(size=(50, 40)), "f32")
    w, _ = stored(rng.normal(size=(40, 30)) / 6, "f32")
    b, _ = stored(rng.normal(size=30), "f32")
    ct, _ = stored(rng.normal(size=(50, 30)), "f32")
    y, z = torch.empty(50, 30, device="cuda"), torch.empty(50, 30, device="cuda")
    ws = scratch(R.psk_linear_workspace(x, w))

    def f(x, w, b):
        R.psk_linear(x, w, y, b, "gelu", z=z, workspace=ws)
        return float((y.double() * ct.double()).sum())

    f(x, w, b)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    R.psk_linear_backward(ct, x, w, dx, dw, db, act="gelu", z=z.clone(),
                          workspace=scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw, db, act="gelu")))
    h = 2.0 ** -6
    for t, g, args in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        v = torch.from_numpy(rng.choice([-1.0, 1.0], size=tuple(t.shape)).astype(np.float32)).cuda() / 8
        at = [[x, w, b], [x, w, b]]
        at[0][args], at[1][args] = t + h * v, t - h * v
        got = (f(*at[0]) - f(*at[1])) / (2 * h)
        want = float((g.double() * v.double()).sum())
        # truncation: h^2 / 6 of the third derivative (below 3 a unit of z), sums of 1500 z's that move by at most 5 v;
        # rounding: 1500 values of f32 off by 1e-6 over 2 h
        assert abs(got - want) < 0.05 + 0.01 * abs(want), (args, got, want)


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph(R):
    rng = np.random.default_rng(9)
    for dtype in ("bf16", "f32"):
        x, _ = stored(rng.normal(size=(600, 520)), dtype)
        w, _ = stored(rng.normal(size=(520, 712)), dtype)
        ct, _ = stored(rng.normal(size=(600, 712)), dtype)
        outs = [[torch.empty(600, 712, device="cuda", dtype=DT[dtype]), torch.empty_like(x), torch.empty_like(w),
                 torch.empty(712, device="cuda")] for _ in range(3)]

        def run(o, stream=None):
            y, dx, dw, db = o[:4]
            ws = o[4:]
            R.psk_linear(x, w, y, act="silu", workspace=ws[0], stream=stream)
            R.psk_linear_backward(ct, x, w, dx, dw, db, act="gelu", z=y, workspace=ws[1], stream=stream)

        for o in outs:
            o += [scratch(R.psk_linear_workspace(x, w)),
                  scratch(R.psk_linear_backward_workspace(ct, x, w, *o[1:4], act="gelu"))]
        run(outs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        run(outs[1], side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(outs[2])
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0][:4], o[:4]))


@pytest.mark.parametrize("rows,cin,cout,dtype,at", [(8, 1024, 640, "bf16", 1), (400, 512, 640, "bf16", 1), (3000, 512, 2048, "bf16", 3),
                                                    (1500, 512, 1000, "bf16", 5), (300, 512, 600, "f32", 1), (1003, 512, 1501, "f32", 3)])
def test_a_lost_copy_ends_in_a_status_not_a_hang(R, rows, cin, cout, dtype, at):
    """In each of the product's kernels: few tiles, pairs of CTAs, single ones; parts of f32 shared and unshared."""
    x = torch.randn(rows, cin, device="cuda").to(DT[dtype])
    w = torch.randn(cin, cout, device="cuda").to(DT[dtype])
    y, ref = (torch.empty(rows, cout, device="cuda", dtype=DT[dtype]) for _ in range(2))
    ws = scratch(R.psk_linear_workspace(x, w))
    R.psk_linear(x, w, ref, workspace=ws)
    assert R.psk_device_status(reset=True) == 0
    try:
        R.psk_test_drop_row(at)
        R.psk_linear(x, w, y, workspace=ws)
        torch.cuda.synchronize()
        assert R.psk_device_status(reset=True) == 1
    finally:
        R.psk_test_drop_row(-1)
    R.psk_linear(x, w, y, workspace=ws)
    torch.cuda.synchronize()
    assert R.psk_device_status() == 0 and torch.equal(y, ref)
