"""f32 products to their last digits in each of the kernels that take them:
operands whose partial sums are exact, so that the tolerance is a few roundings
and every product of parts has to be there once."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.linear_digits import PAIRS, parts, product, tolerance
from tests.train_util import scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _put(p, dtype="f32"):
    """A tensor of the parts' sum, or of the first part alone in bf16, and the parts that it has."""
    t = torch.from_numpy((p.sum(0) if dtype == "f32" else p[0]).astype(np.float32)).cuda()
    return (t, p) if dtype == "f32" else (t.bfloat16(), p[:1])


def _check(got, a, b, terms):
    pairs = [(i, j) for i, j in PAIRS if i < len(a) and j < len(b)]
    want = product(a, b, pairs)
    off = (np.abs(got.double().cpu().numpy() - want) / want).max()
    assert off <= tolerance(terms), (off, tolerance(terms))


# few tiles shared out on 64 and on 128 rows, many tiles, one tile, odd sides
SHAPES = [(64, 512, 128), (300, 1000, 200), (1024, 1024, 1024), (2000, 700, 1500), (100, 200, 90), (509, 771, 1003)]


@pytest.mark.parametrize("rows,cin,cout", SHAPES)
@pytest.mark.parametrize("xt,wt", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_forward(R, rows, cin, cout, xt, wt, layout):
    rng = np.random.default_rng(rows + cin)
    x, xp = _put(parts(rng, (rows, cin), 1.5), xt)
    w, wp = _put(parts(rng, (cin, cout), 1.25), wt)
    w = w if layout == "in_out" else w.t().contiguous().t()
    y = torch.empty(rows, cout, device="cuda")
    R.psk_linear(x, w, y, workspace=scratch(R.psk_linear_workspace(x, w)))
    _check(y, xp, wp, cin)


# both gradients in one launch, each shared out, each over many tiles
@pytest.mark.parametrize("rows,cin,cout", [(300, 200, 104), (509, 771, 1003), (2000, 1500, 1400), (130, 600, 600)])
@pytest.mark.parametrize("types", [("f32", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "f32", "f32")])
def test_backward(R, rows, cin, cout, types):
    rng = np.random.default_rng(rows + cout)
    ct, cp = _put(parts(rng, (rows, cout), 1.5), types[0])
    x, xp = _put(parts(rng, (rows, cin), 1.25), types[1])
    w, wp = _put(parts(rng, (cin, cout), 1.25), types[2])
    dx, dw = torch.empty(rows, cin, device="cuda"), torch.empty(cin, cout, device="cuda")
    R.psk_linear_backward(ct, x, w, dx, dw, None, workspace=scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw)))
    _check(dx, cp, wp.transpose(0, 2, 1), cout)
    _check(dw, xp.transpose(0, 2, 1), cp, rows)


@pytest.mark.parametrize("rows,cin,cout", SHAPES)
def test_normal_values(R, rows, cin, cout):
    """Of normal operands the result is off by less than 2^-20 of its size: sixteen truncated additions a piece, each
    by half a step of 2^-23 of the piece's sum on average at most."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = (torch.randn(*s, generator=g, device="cuda") for s in ((rows, cin), (cin, cout)))
    y = torch.empty(rows, cout, device="cuda")
    R.psk_linear(x, w, y, workspace=scratch(R.psk_linear_workspace(x, w)))
    want = x.double() @ w.double()
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -20
