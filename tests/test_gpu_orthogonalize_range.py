"""psk_orthogonalize of matrices whose squares leave f32, up to f32's largest
values."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_orthogonalize import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


@pytest.mark.parametrize("rows,cols", [(64, 192), (192, 64), (128, 256), (200, 300), (300, 200), (130, 1500)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_elements_up_to_the_largest(R, rows, cols, dtype):
    rng = np.random.default_rng(rows)
    for top in (3.3e38, 1e38, 2.0 ** 120, 2.0 ** 63):
        _run(R, 1, rows, cols, dtype, dtype, eps=0.0, make=lambda: top * rng.uniform(0.25, 1.0, size=(rows, cols))
             * rng.choice([-1.0, 1.0], size=(rows, cols)))


@pytest.mark.parametrize("rows,cols", [(64, 192), (200, 300)])
def test_few_large_elements_among_small_ones(R, rows, cols):
    rng = np.random.default_rng(cols)

    def make():
        v = rng.normal(size=(rows, cols))
        v[:, :5] *= 1e38
        return np.clip(v, -3.3e38, 3.3e38)

    _run(R, 1, rows, cols, "f32", "f32", steps=2, eps=0.0, make=make)
