"""psk_orthogonalize against its binary64 definition.  One step is held to an
elementwise bound of its roundings; for several, the distance from the
definition is compared with the one that the declared roundings of the
iterates make by themselves (the same chain in binary64 with the iterates
rounded as they are stored)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.guard import guarded
from tests.train_util import DT, scratch, stored, strided

pytestmark = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _run(R, n, rows, cols, xt, yt, steps=5, co=MUON, scale=1.0, eps=1e-7, pad=None, make=None, seed=0):
    rng = np.random.default_rng(rows * 3 + cols + seed)
    make = make or (lambda: rng.normal(size=(rows, cols)) * 1e-3)
    xs = [stored(make(), xt) for _ in range(n)]
    ts = [strided(t, *pad) if pad else t for t, _ in xs]
    gs = [guarded((rows, cols), DT[yt]) for _ in range(n)]
    ys = [strided(g.tensor, *pad) if pad else g.tensor for g in gs]
    R.psk_orthogonalize(ts, ys, steps, co, eps, scale, scratch(R.psk_orthogonalize_workspace(n, rows, cols, DT[yt])))
    torch.cuda.synchronize()
    assert all(g.intact() for g in gs)
    triples = [co] * steps if not hasattr(co[0], "__len__") else list(co)
    half, planes = torch.finfo(DT[yt]).eps / 2, 2 if yt == "f32" else 1
    for y, (_, v) in zip(ys, xs):
        got = y.double().cpu().numpy()
        want = OM.orthogonalize(v, triples, steps, eps, scale)
        size = np.linalg.norm(want)
        own = np.linalg.norm(OM.orthogonalize_rounded(v, triples, steps, eps, scale, planes) - want)
        # the roundings' own size twice (other f32 sums flip some of them), the result's storage, and the f32 sums:
        # three products a step, each off by the truncations of its sum and carried on by at most 4
        m = min(rows, cols)
        sums = 4 * 3 * steps * (2.0 ** -24 * 40 if planes == 2 else 17 * 2.0 ** -23 * (max(rows, cols) / 16 + 1) / max(
            1.0, max(rows, cols) ** 0.5))
        assert np.linalg.norm(got - want) <= 2 * own + (half + sums) * size, (
            np.linalg.norm(got - want) / size, own / size, m)


@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 1, 50), (1, 50, 1), (2, 64, 192), (2, 192, 64), (3, 131, 77),
                                         (2, 77, 301), (1, 256, 256), (2, 300, 700), (2, 513, 517), (5, 16, 16),
                                         (1, 128, 1000), (1, 129, 128), (7, 100, 260)])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_against_binary64(R, n, rows, cols, xt, yt):
    _run(R, n, rows, cols, xt, yt)


@pytest.mark.parametrize("rows,cols", [(1024, 1536), (1500, 1024)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_large(R, rows, cols, yt):
    _run(R, 2, rows, cols, yt, yt)


@pytest.mark.parametrize("pad", [(8, 0), (3, 1)])
@pytest.mark.parametrize("rows,cols", [(96, 200), (200, 96), (70, 33)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_strided(R, pad, rows, cols, yt):
    _run(R, 2, rows, cols, yt, yt, pad=pad)


@pytest.mark.parametrize("steps,co,scale", [(1, MUON, 1.0), (2, (1.5, -0.5, 0.0), 0.2), (3, [(4.0, -6.0, 2.5), (3.0, -3.5, 1.2), (
    1.875, -1.25, 0.375)], -3.0), (8, (1.875, -1.25, 0.375), 1.0)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_steps_coefficients_and_scale(R, steps, co, scale, yt):
    _run(R, 2, 90, 160, "f32", yt, steps, co, scale)
    _run(R, 1, 160, 90, "bf16", yt, steps, co, scale)


@pytest.mark.parametrize("rows,cols", [(60, 140), (140, 60), (300, 280)])
def test_one_step_elementwise(R, rows, cols):
    """f32 results: every rounding of one step carried through with magnitudes."""
    rng = np.random.default_rng(7)
    x, v = stored(rng.normal(size=(rows, cols)), "f32")
    y = torch.empty_like(x)
    a, b, c = MUON
    R.psk_orthogonalize([x], [y], 1, MUON, 0.0, 1.0, scratch(R.psk_orthogonalize_workspace(1, rows, cols, torch.float32)))
    X = v.astype(np.float64).T if rows > cols else v.astype(np.float64)
    X = X / np.linalg.norm(X)
    h = 2.0 ** -22                              # two fp16 parts of a value: 2^-11 of the first's 2^-11
    s = OM.sum_error(X.shape[1], True) + 2 * h  # a product's sum, and the product of second parts left out
    Xa = np.abs(X)
    A, B1 = X @ X.T, Xa @ Xa.T
    eX = 4 * h * Xa + 2.0 ** -34                # the norm and the factor, the parts; their smallest step
    eA = s * B1 + 2 * (eX @ Xa.T) + h * B1 + 2.0 ** -34
    B = b * A + c * A @ A
    Ba = abs(b) * np.abs(A) + abs(c) * np.abs(A) @ np.abs(A)
    eB = abs(b) * eA + abs(c) * (2 * np.abs(A) @ eA + s * np.abs(A) @ np.abs(A)) + 2 * h * Ba + 2.0 ** -34
    want = a * X + B @ X
    bound = abs(a) * eX + eB @ Xa + np.abs(B) @ eX + s * np.abs(B) @ Xa + 2 * h * (np.abs(a * X) + np.abs(B) @ Xa)
    got = y.double().cpu().numpy()
    got = got.T if rows > cols else got
    assert (np.abs(got - want) <= 1.1 * bound).all(), (np.abs(got - want) / bound).max()


def test_values_that_a_users_momentum_has(R):
    """Strong directions, rows of very different size, rank below the shorter side, huge and tiny scales."""
    rng = np.random.default_rng(8)
    low = rng.normal(size=(80, 6)) @ rng.normal(size=(6, 200))
    for make in (lambda: low * np.exp(rng.normal(size=(80, 1))), lambda: low * 1e25, lambda: low * 1e-15):
        _run(R, 2, 80, 200, "f32", "f32", make=make, eps=0.0)
        _run(R, 2, 80, 200, "bf16", "bf16", make=make, eps=0.0)


@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_zero_and_broken_matrices_stay_alone(R, yt):
    rng = np.random.default_rng(9)
    xs = [stored(rng.normal(size=(40, 70)), "f32")[0] for _ in range(4)]
    alone = torch.empty(40, 70, device="cuda", dtype=DT[yt])
    R.psk_orthogonalize([xs[3]], [alone], workspace=scratch(R.psk_orthogonalize_workspace(1, 40, 70, DT[yt])))
    xs[0].zero_()
    xs[1][3, 4], xs[2][0, 0] = float("nan"), float("inf")
    ys = [torch.empty(40, 70, device="cuda", dtype=DT[yt]) for _ in range(4)]
    R.psk_orthogonalize(xs, ys, workspace=scratch(R.psk_orthogonalize_workspace(4, 40, 70, DT[yt])))
    assert not bool(ys[0].any()) and bool(ys[1].isnan().all()) and bool(ys[2].isnan().all())
    assert torch.equal(ys[3], alone)


@pytest.mark.parametrize("rows,cols", [(64, 192), (200, 130), (700, 300)])
def test_in_place_swapped_and_in_a_graph(R, rows, cols):
    rng = np.random.default_rng(10)
    base = [stored(rng.normal(size=(rows, cols)), "bf16")[0] for _ in range(2)]
    want = [torch.empty_like(b) for b in base]
    ws = [scratch(R.psk_orthogonalize_workspace(2, rows, cols, torch.bfloat16)) for _ in range(2)]
    R.psk_orthogonalize(base, want, workspace=ws[0])
    xs = [b.clone() for b in base]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    R.psk_orthogonalize(xs, [xs[1], xs[0]], workspace=ws[1], stream=side)      # each into the other's place
    side.synchronize()
    assert torch.equal(xs[1], want[0]) and torch.equal(xs[0], want[1])
    xs = [b.clone() for b in base]
    graph = torch.cuda.CUDAGraph()
    ys = [torch.empty_like(b) for b in base]
    with torch.cuda.graph(graph):
        R.psk_orthogonalize(xs, ys, workspace=ws[1])
    for x in xs:
        x.copy_(base[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[0])


def test_nothing_to_do(R):
    R.psk_orthogonalize([], [])
    e = torch.empty(0, 5, device="cuda")
    R.psk_orthogonalize([e], [e])
