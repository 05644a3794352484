"""Products whose tiles are shared out among the CTAs of a cluster, with sides
that leave the lanes of a warp different numbers of elements before the
cluster's barriers, many times over."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.train_util import DT, close, scratch, stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cin,cout", [(1, 515, 1), (3, 1000, 130), (7, 2048, 333), (33, 640, 129), (65, 1100, 257),
                                           (131, 900, 131), (200, 3000, 77)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_sides(rows, cin, cout, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    rng = np.random.default_rng(rows)
    x, xv = stored(rng.normal(size=(rows, cin)), dtype)
    w, wv = stored(rng.normal(size=(cin, cout)) / cin ** 0.5, dtype)
    ct, cv = stored(rng.normal(size=(rows, cout)), dtype)
    y, dx, dw = (torch.empty(s, device="cuda", dtype=DT[dtype]) for s in ((rows, cout), (rows, cin), (cin, cout)))
    db = torch.empty(cout, device="cuda")
    ws = scratch(R.psk_linear_workspace(x, w))
    wb = scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw, db))
    first = None
    for _ in range(40):
        R.psk_linear(x, w, y, workspace=ws)
        R.psk_linear_backward(ct, x, w, dx, dw, db, workspace=wb)
        out = [t.clone() for t in (y, dx, dw, db)]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    assert R.psk_device_status() == 0
    for got, a, b in ((y, xv, wv), (dx, cv, wv.T), (dw, xv.T, cv)):
        (want, err), _ = OM.linear(a, b, None, "none", None, dtype == "f32")
        close(got, want, err, dtype)
    close(db, cv.astype(np.float64).sum(0), (rows + 4) * 2.0 ** -24 * np.abs(cv.astype(np.float64)).sum(0), "f32")
