"""Long sums of bf16 products whose result is f32, all terms of one sign (a
truncation's errors then add up): a leaf's gradient over many tokens, results
of wide layers."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.train_util import DT, close, scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _positive(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (0.5 + torch.rand(*shape, generator=g, device="cuda")).bfloat16()


def _near(got, want, terms):
    """Up to 2048 terms the tensor core adds, sixteen at a time; beyond, it adds pieces of 1024.  Each of its additions
    truncates by about a step (2^-23) of a partial sum that is half the whole on average; the pieces are added with one
    rounding each (half a step of a running sum)."""
    pieces = -(-terms // 1024) if terms > 2048 else 1
    bound = min(terms, 1024 if pieces > 1 else 2048) / 16 * 2.0 ** -23 + (pieces / 2 + 10) * 2.0 ** -24
    err = ((got.double() - want) / want).abs().max().item()
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("rows,cin,cout", [(16384, 64, 128), (65536, 64, 72), (32768, 300, 520), (20000, 1033, 2048),
                                           (65536, 2048, 2816)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_f32_leaf_of_a_bf16_layer(R, rows, cin, cout, accumulate):
    x, ct, w = _positive(1, rows, cin), _positive(2, rows, cout), _positive(3, cin, cout)
    dw = torch.full((cin, cout), 7.0, device="cuda")
    want = x.double().t() @ ct.double() + (7.0 if accumulate else 0.0)
    for dx in (None, torch.empty_like(x)):
        dw.fill_(7.0)
        R.psk_linear_backward(ct, x, w, dx, dw, None, accumulate=accumulate,
                              workspace=scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw)))
        _near(dw, want, rows)
        if dx is not None:
            close(dx[:64], (ct[:64].double() @ w.double().t()).cpu().numpy(), 1e-4 * cout, "bf16")


@pytest.mark.parametrize("rows,cin,cout", [(8, 16384, 256), (20, 16384, 512), (50, 8192, 1000), (700, 8192, 1024),
                                           (2000, 4096, 2056), (4096, 2048, 4096),
                                           (1000, 2049, 3000)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_f32_results(R, rows, cin, cout, layout):
    x, w = _positive(4, rows, cin), _positive(5, cin, cout)
    w = w if layout == "in_out" else w.t().contiguous().t()
    want = x.double() @ w.double()
    y, z = torch.empty(rows, cout, device="cuda"), torch.empty(rows, cout, device="cuda")
    ws = scratch(R.psk_linear_workspace(x, w))
    R.psk_linear(x, w, y, workspace=ws)
    _near(y, want, cin)
    y16 = torch.empty(rows, cout, device="cuda", dtype=DT["bf16"])
    R.psk_linear(x, w, y16, act="silu", z=z, workspace=ws)               # z f32, y bf16
    _near(z, want, cin)
    dx = torch.empty(rows, cin, device="cuda")
    R.psk_linear_backward(y16, x, w, dx, None, None,
                          workspace=scratch(R.psk_linear_backward_workspace(y16, x, w, dx)))
    _near(dx, y16.double() @ w.double().t(), cout)


@pytest.mark.parametrize("rows,cin,cout", [(300, 1 << 19, 128), (16, 1 << 19, 64), (1500, 1 << 18, 1300)])
def test_bf16_results_of_very_long_sums(R, rows, cin, cout):
    """Beyond 2^16 terms truncations would pass bf16's own rounding by and by."""
    x, w = _positive(6, rows, cin), _positive(7, cin, cout)
    y = torch.empty(rows, cout, device="cuda", dtype=DT["bf16"])
    R.psk_linear(x, w, y, workspace=scratch(R.psk_linear_workspace(x, w)))
    want = x.double() @ w.double()
    err = ((y.double() - want) / want).abs().max().item()
    assert err <= 2.0 ** -8 + 64 * 2.0 ** -23 + (cin / 2048 + 10) * 2.0 ** -24, err


@pytest.mark.parametrize("dwt", ["f32", "bf16"])
def test_both_gradients_of_one_launch(R, dwt):
    rows, cin, cout = 2688, 512, 2176
    x, ct, w = _positive(8, rows, cin), _positive(9, rows, cout), _positive(10, cin, cout)
    dx, dw = torch.empty(rows, cin, device="cuda"), torch.empty(cin, cout, device="cuda", dtype=DT[dwt])
    R.psk_linear_backward(ct, x, w, dx, dw, None, workspace=scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw)))
    _near(dx, ct.double() @ w.double().t(), cout)
    want = x.double().t() @ ct.double()
    if dwt == "f32":
        _near(dw, want, rows)
    else:
        close(dw, want.cpu().numpy(), want.cpu().numpy() * (rows / 16) * 2.0 ** -23, "bf16")


@pytest.mark.parametrize("n,rows,cols", [(80, 16, 70000), (2, 64, 600000), (1, 300000, 130)])
def test_updates_of_very_long_matrices(R, n, rows, cols):
    from tests.test_gpu_orthogonalize import _run

    _run(R, n, rows, cols, "bf16", "bf16")
