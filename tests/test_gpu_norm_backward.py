"""psk_norm_backward against its binary64 definition, within the bounds that
f32 sums and the storage roundings keep."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.training as OT
from tests.guard import guarded
from tests.train_util import DT, close, scratch, stored, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


EPS = {"rms": 1e-6, "layer": 1e-5}


def _check(R, kind, rows, cols, xt, ct_t, dxt, pt, gt, mean=0.25, pad=None, inplace=None, seed=0):
    rng = np.random.default_rng(rows * 7 + cols + seed)
    x, xv = stored(rng.normal(size=(rows, cols)) + mean, xt)
    c, cv = stored(rng.normal(size=(rows, cols)), ct_t)
    gamma, gv = stored(1 + 0.1 * rng.normal(size=cols), pt) if pt else (None, None)
    if pad:
        x, c = strided(x, *pad), strided(c, *pad)
    go = guarded((rows, cols), DT[dxt])
    dx = {"x": x, "ct": c, None: go.tensor}[inplace]
    if pad and not inplace:
        dx = strided(dx, *pad)
    dg, db = guarded((cols,), DT[gt]), guarded((cols,), DT[gt])
    ws = scratch(R.psk_norm_backward_workspace(rows, cols))
    R.psk_norm_backward(x, c, dx, kind, EPS[kind], gamma, dg.tensor, db.tensor if kind == "layer" else None, ws)
    torch.cuda.synchronize()
    assert go.intact() and dg.intact() and db.intact()
    (wx, ex), (wg, eg), (wb, eb) = OT.norm_backward(xv, cv, gv, kind, EPS[kind])
    close(dx, wx, ex, dxt)
    close(dg.tensor, wg, eg, gt)
    if kind == "layer":
        close(db.tensor, wb, eb, gt)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (3, 5), (64, 64), (100, 65), (7, 771), (37, 1000), (200, 512),
                                       (65, 2048), (40, 4096), (33, 8192), (9, 16384), (5, 10000), (3, 49152),
                                       (1000, 8), (2, 4104)])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16", "bf16", "f32"), ("f32", "f32", "f32", "f32", "f32")],
                         ids=["bf16", "f32"])
def test_against_binary64(R, kind, rows, cols, types):
    _check(R, kind, rows, cols, *types)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("types", [("bf16", "f32", "bf16", "f32", "bf16"), ("f32", "bf16", "bf16", None, "bf16"),
                                   ("bf16", "bf16", "f32", "f32", "f32"), ("f32", "f32", "bf16", "bf16", "f32")])
@pytest.mark.parametrize("rows,cols", [(50, 256), (19, 333), (12, 2056)])
def test_mixed_types(R, kind, rows, cols, types):
    _check(R, kind, rows, cols, *types)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("inplace", [None, "x", "ct"])
@pytest.mark.parametrize("cols,pad", [(256, (8, 8)), (256, (3, 1)), (131, (5, 0)), (4096, (8, 0)), (12288, (8, 0))])
def test_strided_and_in_place(R, kind, inplace, cols, pad):
    _check(R, kind, 45, cols, "bf16", "bf16", "bf16", "bf16", "f32", pad=pad, inplace=inplace)


@pytest.mark.parametrize("rows,cols", [(3000, 256), (300, 1024)])
def test_a_large_mean_keeps_the_layer_norms_digits(R, rows, cols):
    _check(R, "layer", rows, cols, "f32", "f32", "f32", "f32", "f32", mean=50.0)


def test_no_rows_give_zero_parameter_gradients(R):
    x = torch.empty(0, 77, device="cuda")
    dg, db = torch.full((77,), float("nan"), device="cuda"), torch.full((77,), float("nan"), device="cuda")
    R.psk_norm_backward(x, x, x, "layer", 1e-5, None, dg, db)
    assert not bool(dg.any()) and not bool(db.any())


@pytest.mark.parametrize("want", ["none", "dgamma", "dbeta"])
def test_unwanted_parameter_gradients(R, want):
    rng = np.random.default_rng(1)
    x, xv = stored(rng.normal(size=(70, 264)), "bf16")
    c, cv = stored(rng.normal(size=(70, 264)), "bf16")
    dx, out = torch.empty(70, 264, device="cuda"), guarded((264,), torch.float32)
    ws = scratch(R.psk_norm_backward_workspace(70, 264))
    R.psk_norm_backward(x, c, dx, "layer", 1e-5, None, out.tensor if want == "dgamma" else None,
                        out.tensor if want == "dbeta" else None, ws)
    res = OT.norm_backward(xv, cv, None, "layer", 1e-5)
    close(dx, *res[0], "f32")
    if want != "none":
        close(out.tensor, *res[1 if want == "dgamma" else 2], "f32")
    else:
        assert bool(out.tensor.isnan().all())


def test_a_nan_row_stays_in_its_row(R):
    rng = np.random.default_rng(2)
    x, xv = stored(rng.normal(size=(20, 512)), "f32")
    c, cv = stored(rng.normal(size=(20, 512)), "f32")
    x[4, 9] = float("nan")
    dx = torch.empty_like(x)
    R.psk_norm_backward(x, c, dx, "rms", 1e-6, workspace=scratch(R.psk_norm_backward_workspace(20, 512)))
    assert bool(dx[4].isnan().all()) and not bool(dx[torch.arange(20) != 4].isnan().any())


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph(R):
    rng = np.random.default_rng(3)
    x, _ = stored(rng.normal(size=(600, 1024)), "bf16")
    c, _ = stored(rng.normal(size=(600, 1024)), "bf16")
    outs = []
    for _ in range(3):
        outs.append((torch.empty_like(x), torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda"),
                     scratch(R.psk_norm_backward_workspace(600, 1024))))
    dx, dg, db, ws = outs[0]
    R.psk_norm_backward(x, c, dx, "layer", 1e-5, None, dg, db, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dx, dg, db, ws = outs[1]
    R.psk_norm_backward(x, c, dx, "layer", 1e-5, None, dg, db, ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    dx, dg, db, ws = outs[2]
    with torch.cuda.graph(graph):
        R.psk_norm_backward(x, c, dx, "layer", 1e-5, None, dg, db, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0][:3], o[:3]))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,cols,dtype", [(2000, 4096, "bf16"), (3000, 2048, "f32"), (1500, 1032, "bf16"),
                                             (700, 16384, "bf16"), (900, 12288, "f32"), (1100, 8192, "bf16"),
                                             (4000, 320, "bf16"), (2500, 1001, "f32")])
def test_many_rows(R, kind, rows, cols, dtype):
    _check(R, kind, rows, cols, dtype, dtype, dtype, dtype, "f32")


def test_a_lost_copy_ends_in_a_status_not_a_hang(R):
    x = torch.randn(900, 4096, device="cuda", dtype=torch.bfloat16)
    dx, dg = torch.empty_like(x), torch.empty(4096, device="cuda")
    ws = scratch(R.psk_norm_backward_workspace(900, 4096))
    assert R.psk_device_status(reset=True) == 0
    try:
        R.psk_test_drop_row(3)
        R.psk_norm_backward(x, x, dx, "rms", 1e-6, None, dg, workspace=ws)
        torch.cuda.synchronize()
        assert R.psk_device_status(reset=True) == 1
    finally:
        R.psk_test_drop_row(-1)
    R.psk_norm_backward(x, x, dx, "rms", 1e-6, None, dg, workspace=ws)
    torch.cuda.synchronize()
    assert R.psk_device_status() == 0 and bool(dx.isfinite().all()) and bool(dg.isfinite().all())
