"""psk_dropout against the oracle, bit for bit (one f32 rounding per
operation, the generator's words exactly)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.training as OT
from tests.guard import guarded
from tests.train_util import DT, same_bits, stored, strided

pytestmark = pytest.mark.gpu
SEED = 0x9E3779B97F4A7C15


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (5, 7), (2, 8), (127, 1003), (64, 64), (1, 4099), (300, 20),
                                       (9, 4096)])
@pytest.mark.parametrize("xt,rt,yt", [("f32", None, "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                      ("f32", "bf16", "bf16"), ("bf16", None, "f32")])
@pytest.mark.parametrize("p,offset", [(0.1, 0), (0.5, (1 << 40) + 3)])
def test_bitwise(R, rows, cols, xt, rt, yt, p, offset):
    rng = np.random.default_rng(rows + cols)
    x, xv = stored(rng.normal(size=(rows, cols)), xt)
    r, rv = stored(rng.normal(size=(rows, cols)), rt) if rt else (None, None)
    g = guarded((rows, cols), DT[yt])
    R.psk_dropout(x, g.tensor, p, SEED, offset, residual=r)
    torch.cuda.synchronize()
    assert g.intact()
    same_bits(g.tensor, OT.dropout(xv, rv, p, SEED, offset), yt)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -33, 2.0 ** -32, 1e-4, 1 - 2.0 ** -32, 1 - 2.0 ** -34, 1.0])
def test_probabilities_at_the_ends(R, p):
    x, xv = stored(np.random.default_rng(1).normal(size=(16, 1000)), "f32")
    y = torch.empty_like(x)
    R.psk_dropout(x, y, p, 5)
    same_bits(y, OT.dropout(xv, None, p, 5, 0), "f32")


def test_dropped_elements_never_reach_the_result(R):
    keep = OT.dropout_keep(8, 64, 0.5, 3, 0)
    xv = np.where(keep, 1.0, np.resize([np.nan, np.inf, -np.inf], (8, 64))).astype(np.float32)
    x = torch.from_numpy(xv).cuda()
    y = torch.empty_like(x)
    R.psk_dropout(x, y, 0.5, 3)
    assert np.array_equal(y.cpu().numpy(), np.where(keep, 2.0, 0.0))
    R.psk_dropout(torch.full_like(x, float("nan")), y, 1.0, 3)
    assert not bool(y.any())


def test_the_backward_draws_the_forwards_mask(R):
    x = torch.ones(37, 130, dtype=torch.bfloat16, device="cuda")
    ct = torch.full((37, 130 + 6), 3.0, device="cuda")[:, 3:133]      # other type, other strides
    y, dx = torch.empty_like(x), torch.empty(37, 130, device="cuda")
    R.psk_dropout(x, y, 0.25, 11, 12)
    R.psk_dropout(ct, dx, 0.25, 11, 12)
    assert torch.equal(y != 0, dx != 0) and set(dx.unique().tolist()) == {0.0, 4.0}


@pytest.mark.parametrize("cols,pad,offset", [(64, 8, 8), (64, 3, 1), (61, 3, 0)])
@pytest.mark.parametrize("target", ["x", "residual"])
def test_in_place_and_strided(R, cols, pad, offset, target):
    rng = np.random.default_rng(2)
    (x, xv), (r, rv) = stored(rng.normal(size=(50, cols)), "bf16"), stored(rng.normal(size=(50, cols)), "bf16")
    x, r = strided(x, pad, offset), strided(r, pad, offset)
    R.psk_dropout(x, x if target == "x" else r, 0.3, 1, 2, residual=r)
    same_bits((x if target == "x" else r).contiguous(), OT.dropout(xv, rv, 0.3, 1, 2), "bf16")


def test_vectors_are_one_row(R):
    x, xv = stored(np.random.default_rng(3).normal(size=(1, 515)), "f32")
    y = torch.empty(515, device="cuda")
    R.psk_dropout(x[0], y, 0.2, 9)
    same_bits(y[None], OT.dropout(xv, None, 0.2, 9, 0), "f32")


def test_counter_gives_captured_replays_new_masks(R):
    x, xv = stored(np.random.default_rng(4).normal(size=(20, 72)), "f32")
    y, counter = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device="cuda")
    R.psk_dropout(x, y, 0.4, 21, 7, counter=counter)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.psk_dropout(x, y, 0.4, 21, 7, counter=counter)
        counter.add_(1)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        same_bits(y, OT.dropout(xv, None, 0.4, 21, 7 + step), "f32")
    counter.fill_(-8)                                   # added mod 2^64
    graph.replay()
    torch.cuda.synchronize()
    same_bits(y, OT.dropout(xv, None, 0.4, 21, (7 - 8) % (1 << 64)), "f32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    R.psk_dropout(x, y, 0.4, 21, 3, stream=side)
    side.synchronize()
    same_bits(y, OT.dropout(xv, None, 0.4, 21, 3), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1, 3, 9, 65, 1001, 1002, 1004])
@pytest.mark.parametrize("start,pad", [(0, 0), (1, 0), (3, 5), (5, 2), (7, 1)])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_beginning_anywhere(R, dtype, cols, start, pad, residual):
    """x, y and the residual alike, at every distance from a 16-byte boundary, neighbours untouched."""
    rng = np.random.default_rng(cols + start)
    rows, ld = 11, cols + pad

    def make():
        t, v = stored(rng.normal(size=(rows, cols)), dtype)
        buf = torch.full((start + rows * ld + 16,), 7.0, dtype=DT[dtype], device="cuda")
        view = buf[start:start + rows * ld].view(rows, ld)[:, :cols]
        view.copy_(t)
        return buf, view, v

    (_, x, xv), (_, r, rv), (buf, y, _) = make(), make(), make()
    y.fill_(float("nan"))
    R.psk_dropout(x, y, 0.4, 99, 3, residual=r if residual else None)
    same_bits(y.contiguous(), OT.dropout(xv, rv if residual else None, 0.4, 99, 3), dtype)
    y.fill_(7.0)
    assert bool((buf == 7.0).all())
