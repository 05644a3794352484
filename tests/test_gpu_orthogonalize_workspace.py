"""psk_orthogonalize with a workspace on any 16-byte boundary."""

import pytest

torch = pytest.importorskip("torch")

from tests.train_util import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,rows,cols", [(2, 200, 300), (1, 300, 140), (3, 64, 1000), (2, 600, 700), (2, 64, 192)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_workspace_on_any_16_byte_boundary(n, rows, cols, dtype):
    """The same bits from each, nothing written beside it; in place into each other too."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    g = torch.Generator(device="cuda").manual_seed(rows)
    base = [torch.randn(rows, cols, generator=g, device="cuda").to(DT[dtype]) for _ in range(n)]
    need = R.psk_orthogonalize_workspace(n, rows, cols, DT[dtype])
    want = None
    for at in (0, 16, 32, 48, 112):
        pool = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        assert pool.data_ptr() % 256 == 0
        xs = [b.clone() for b in base]
        R.psk_orthogonalize(xs, xs[1:] + xs[:1], workspace=pool[at:at + need])
        want = want or [x.clone() for x in xs]
        assert all(torch.equal(a, b) for a, b in zip(xs, want))
        assert bool((pool[:at] == 0xA5).all()) and bool((pool[at + need:] == 0xA5).all())
