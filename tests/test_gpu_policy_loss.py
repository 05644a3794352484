"""psk_token_logp and psk_policy_loss against their binary64 definitions, within
the bounds that f32 exponentials and sums and the storage roundings keep."""

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


def _inputs(rng, rows, cols, lt, scale, it="i64"):
    x, xv = stored(rng.normal(size=(rows, cols)) * 2.5, lt)
    t = rng.integers(0, cols, rows)
    t[rng.random(rows) < 0.1] = -1
    t[rng.random(rows) < 0.05] = cols
    if it == "i64":
        t[rng.random(rows) < 0.05] = 1 << 40
    logp = OT.token_logp(xv, t, scale)[0]
    # ratios on both sides of the bounds 0.8 and 1.25, at least 2 % away from them
    old = (logp - np.log(rng.choice([0.3, 0.7, 0.78, 0.82, 1.0, 1.2, 1.28, 2.0], rows))).astype(np.float32)
    ref = (logp + rng.normal(size=rows) * rng.choice([1e-3, 0.3, 2.0], rows)).astype(np.float32)
    adv = rng.normal(size=rows).astype(np.float32)
    adv[rng.random(rows) < 0.1] = 0.0
    w = rng.uniform(0.1, 1.0, rows).astype(np.float32)
    w[rng.random(rows) < 0.15] = 0.0
    targets = torch.from_numpy(t.astype(np.int64 if it == "i64" else np.int32)).cuda()
    return x, xv, t, targets, old, ref, adv, w


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


SHAPES = [(1, 1), (1, 2), (3, 7), (61, 92), (40, 1003), (17, 1024), (9, 5000), (20, 32000), (300, 264), (5, 50001),
          (3, 131072), (2, 300000), (2, 300001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("lt,it", [("f32", "i32"), ("bf16", "i64")])
def test_token_logp(R, rows, cols, lt, it):
    rng = np.random.default_rng(rows + cols)
    x, xv, t, targets, *_ = _inputs(rng, rows, cols, lt, 1.25, it)
    g = guarded((rows,), torch.float32)
    R.psk_token_logp(x, targets, g.tensor, scale=1.25)
    torch.cuda.synchronize()
    assert g.intact()
    want, bound, _, _ = OT.token_logp(xv, t, 1.25)
    close(g.tensor, want, bound, "f32")


def _check(R, rows, cols, lt, gt, kl, scale, uniform=False, grad=True, pad=None, inplace=False, it="i64", seed=0):
    rng = np.random.default_rng(rows * 3 + cols + seed)
    x, xv, t, targets, old, ref, adv, w = _inputs(rng, rows, cols, lt, scale, it)
    if uniform:
        w = None
    if kl is None:
        ref = None
    if pad:
        x = strided(x, *pad)
    loss, logp = guarded((2,), torch.float32), guarded((rows,), torch.float32)
    gg = guarded((rows, cols), DT[gt]) if grad else None
    d = x if inplace else gg.tensor if grad else None
    if pad and grad and not inplace:
        d = strided(d, *pad)
    ws = scratch(R.psk_policy_loss_workspace(rows, cols))
    R.psk_policy_loss(x, targets, _dev(old), _dev(adv), _dev(w), loss.tensor, logp.tensor, d, ref_logp=_dev(ref),
                      clip_low=0.2, clip_high=0.25, kl_coef=kl or 0.0, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    assert loss.intact() and logp.intact() and (gg is None or gg.intact())
    want = OT.policy_loss(xv, t, old, ref, adv, w, 0.2, 0.25, kl or 0.0, scale)
    close(loss.tensor, *want["loss"], "f32")
    close(logp.tensor, *want["logp"], "f32")
    if grad:
        close(d, *want["dlogits"], gt)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("lt,gt,kl,scale", [("f32", "f32", 0.1, 1.0), ("bf16", "bf16", 0.05, 1.25),
                                            ("bf16", "bf16", None, 0.8)])
def test_loss_and_gradient(R, rows, cols, lt, gt, kl, scale):
    _check(R, rows, cols, lt, gt, kl, scale)


@pytest.mark.parametrize("rows,cols", [(30, 2000), (11, 777)])
@pytest.mark.parametrize("lt,gt", [("bf16", "f32"), ("f32", "bf16")])
def test_mixed_types_uniform_weights(R, rows, cols, lt, gt):
    _check(R, rows, cols, lt, gt, 0.2, 1.0, uniform=True, it="i32")


@pytest.mark.parametrize("rows,cols", [(61, 92), (20, 32000), (9, 5001)])
@pytest.mark.parametrize("lt", ["bf16", "f32"])
def test_the_loss_alone(R, rows, cols, lt):
    _check(R, rows, cols, lt, lt, 0.1, 1.0, grad=False)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("cols,pad", [(512, (8, 8)), (512, (3, 1)), (515, (5, 0)), (32000, (8, 0)), (150000, (8, 0))])
def test_strided_and_in_place(R, cols, pad, inplace):
    _check(R, 12, cols, "bf16", "bf16", 0.1, 1.0, pad=pad, inplace=inplace)


def test_many_short_rows(R):
    _check(R, 5000, 40, "f32", "f32", 0.1, 1.0)
    _check(R, 3000, 92, "bf16", "bf16", 0.1, 1.0)


def _plain(R, x, t, old, adv, w, **kw):
    rows, cols = x.shape
    loss, logp, d = torch.empty(2, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    R.psk_policy_loss(x, t, old, adv, w, loss, logp, d, workspace=scratch(R.psk_policy_loss_workspace(rows, cols)), **kw)
    return loss, logp, d


@pytest.mark.parametrize("cols", [1000, 1001, 32000])
def test_rows_left_out_are_not_read(R, cols):
    x = torch.randn(6, cols, device="cuda")
    x[1], x[4] = float("nan"), float("inf")
    t = torch.tensor([3, 5, -1, 0, cols, cols - 1], device="cuda")
    w = torch.tensor([0.5, 0.0, 0.5, 0.25, 0.5, 0.0], device="cuda")
    one = torch.ones(6, device="cuda")
    old = torch.full((6,), -5.0, device="cuda")
    old[1] = float("nan")
    loss, logp, d = _plain(R, x, t, old, one, w, ref_logp=old, kl_coef=0.1)
    assert bool(loss.isfinite().all()) and not bool(logp[[1, 2, 4, 5]].any()) and not bool(d[[1, 2, 4, 5]].any())
    assert bool(d[[0, 3]].any(1).all())
    loss, logp, d = _plain(R, x, t, old, one, torch.zeros(6, device="cuda"), ref_logp=old, kl_coef=0.1)
    assert not bool(loss.any()) and not bool(logp.any()) and not bool(d.any())


@pytest.mark.parametrize("cols", [700, 32000])
@pytest.mark.parametrize("lt", ["f32", "bf16"])
def test_infinite_and_nan_logits(R, cols, lt):
    x = torch.randn(7, cols, device="cuda").to(DT[lt])
    x[0, : cols // 2] = float("-inf")             # refused tokens: probability 0
    x[1] = float("-inf")                          # nothing allowed
    x[2, 9] = float("nan")
    x[3, 9] = float("inf")
    x[4, 0] = float("-inf")                       # the target itself refused
    x[5] = torch.finfo(DT[lt]).min                # every logit the type's lowest value: uniform
    x[6, 1:] = torch.finfo(DT[lt]).min            # one certain token
    t = torch.tensor([cols - 1, 5, 5, 5, 0, 7, 0], device="cuda")
    old = torch.full((7,), -4.0, device="cuda")
    loss, logp, d = _plain(R, x, t, old, torch.ones(7, device="cuda"), None)
    want = torch.log_softmax(x.double(), 1)[torch.arange(7), t]
    assert bool(logp[1:4].isnan().all()) and bool(d[1:4].isnan().all(1).all()) and bool(loss.isnan()[0])
    assert logp[4] == float("-inf") and not bool(d[4].any())
    ok = [0, 5, 6]
    assert torch.allclose(logp[ok].double(), want[ok], rtol=0, atol=5e-6)
    assert bool(d[ok].isfinite().all()) and not bool(d[0, : cols // 2].any()) and not bool(d[6].any())


def test_extreme_ratios(R):
    x = torch.zeros(4, 64, device="cuda")         # logp = -log 64
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    old = torch.tensor([-200.0, -200.0, 200.0, -200.0], device="cuda")
    adv = torch.tensor([1.0, 0.0, 1.0, 0.0], device="cuda")
    loss, logp, d = _plain(R, x, t, old, adv, torch.ones(4, device="cuda"))
    assert abs(float(loss[0]) + 1.2) < 1e-6 and not bool(d.any())   # -1.2 (clipped), 0, ~0, 0


def test_no_rows_give_a_zero_loss(R):
    loss = torch.full((2,), float("nan"), device="cuda")
    e = torch.empty(0, device="cuda")
    R.psk_policy_loss(torch.empty(0, 10, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), e, e, e, loss)
    assert not bool(loss.any())


@pytest.mark.parametrize("cols", [1003, 32000, 131072])
def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph(R, cols):
    rng = np.random.default_rng(3)
    rows = 40
    x, xv, t, targets, old, ref, adv, w = _inputs(rng, rows, cols, "bf16", 1.0)
    old, ref, adv, w = map(_dev, (old, ref, adv, w))

    def bufs():
        return (torch.empty(2, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x),
                scratch(R.psk_policy_loss_workspace(rows, cols)))

    def call(b, stream=None):
        R.psk_policy_loss(x, targets, old, adv, w, b[0], b[1], b[2], ref_logp=ref, kl_coef=0.1, workspace=b[3],
                          stream=stream)

    first, second, third = bufs(), bufs(), bufs()
    call(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(second, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(third)
    graph.replay()
    torch.cuda.synchronize()
    for o in (second, third):
        assert all(torch.equal(a, b) for a, b in zip(first[:3], o[:3]))
    assert R.psk_device_status() == 0


@pytest.mark.parametrize("rows,cols,lt", [(700, 32000, "bf16"), (500, 20001, "bf16"), (2000, 3000, "bf16"),
                                          (400, 33000, "f32"), (900, 9000, "f32")])
def test_many_rows_a_cta(R, rows, cols, lt):
    _check(R, rows, cols, lt, lt, 0.1, 1.0)


@pytest.mark.parametrize("rows,cols,lt", [(200, 131072, "bf16"), (90, 100003, "f32"), (130, 50000, "bf16")])
def test_many_rows_a_cluster(R, rows, cols, lt):
    _check(R, rows, cols, lt, lt, 0.1, 1.0)
    rng = np.random.default_rng(1)
    x, xv, t, targets, *_ = _inputs(rng, rows, cols, lt, 1.0)
    logp = torch.empty(rows, device="cuda")
    R.psk_token_logp(x, targets, logp)
    want, bound, _, _ = OT.token_logp(xv, t, 1.0)
    close(logp, want, bound, "f32")


@pytest.mark.parametrize("rows,cols", [(400, 32000), (100, 131072)])
def test_a_lost_copy_ends_in_a_status_not_a_hang(R, rows, cols):
    x = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16)
    t, logp = torch.zeros(rows, dtype=torch.int64, device="cuda"), torch.empty(rows, device="cuda")
    assert R.psk_device_status(reset=True) == 0
    try:
        R.psk_test_drop_row(1)
        R.psk_token_logp(x, t, logp)
        torch.cuda.synchronize()
        assert R.psk_device_status(reset=True) == 1
    finally:
        R.psk_test_drop_row(-1)
    R.psk_token_logp(x, t, logp)
    torch.cuda.synchronize()
    assert R.psk_device_status() == 0 and bool(logp.isfinite().all())


@pytest.mark.parametrize("rows,cols,lt", [(1200, 20000, "bf16"), (4000, 3001, "bf16"), (1000, 9000, "f32"),
                                          (6000, 500, "f32"), (3000, 6000, "bf16")])
def test_many_rows_without_a_gradient(R, rows, cols, lt):
    _check(R, rows, cols, lt, lt, 0.1, 1.0, grad=False)
    rng = np.random.default_rng(2)
    x, xv, t, targets, *_ = _inputs(rng, rows, cols, lt, 0.8)
    logp = torch.empty(rows, device="cuda")
    R.psk_token_logp(x, targets, logp, scale=0.8)
    want, bound, _, _ = OT.token_logp(xv, t, 0.8)
    close(logp, want, bound, "f32")
