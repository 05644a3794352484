"""What the header states about psk_orthogonalize's accuracy, on matrices of
full rank (all directions of a size: the roundings' effect is largest)."""

import pytest

torch = pytest.importorskip("torch")

from tests.train_util import DT, scratch

pytestmark = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)


def _definition(g):
    x = g.double()
    x = x / (x.norm() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    a, b, c = MUON
    for _ in range(5):
        q = x @ x.t()
        x = a * x + (b * q + c * (q @ q)) @ x
    return x.t() if tall else x


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 2), (4, 30), (16, 16), (40, 300), (64, 64), (64, 192), (192, 64), (128, 256),
                                       (100, 1000), (256, 256), (300, 1024), (512, 2048), (1024, 1024), (2048, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gaussian_matrices(rows, cols, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    limit = 1e-5 if dtype == "f32" else 5e-3 if min(rows, cols) >= 64 else 2e-2
    n = 20 if rows <= 300 else 2
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    xs = [torch.randn(rows, cols, generator=g, device="cuda").to(DT[dtype]) for _ in range(n)]
    ys = [torch.empty_like(x) for x in xs]
    R.psk_orthogonalize(xs, ys, workspace=scratch(R.psk_orthogonalize_workspace(n, rows, cols, DT[dtype])))
    for x, y in zip(xs, ys):
        want = _definition(x)
        assert float((y.double() - want).norm() / want.norm()) <= limit


@pytest.mark.parametrize("co", [[(7.9, 0.0, 0.0), (0.1, 0.0, 0.0)], [(-7.9, 0.0, 0.0), (1.0, -1.0 / 64, 0.0)],
                                [(2.5, 0.0, 0.0), (0.5, 0.25, 1.5)]])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 50), (1, 700), (2, 200)])
def test_singular_values_up_to_the_stated_limit(co, rows, cols):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R
    from tests.test_gpu_orthogonalize import _run

    _run(R, 2, rows, cols, "f32", "f32", len(co), co)
