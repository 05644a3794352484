"""psk_token_logp and psk_policy_loss at the ends of their range, against the
binary64 definitions: targets at a mask's fill, differences and products that
leave f32's range."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.training as OT
from tests.train_util import DT, close, scratch, stored

pytestmark = pytest.mark.gpu

# One CTA's rows (aligned, and beginning anywhere), a cluster's, and rows beyond a cluster.
COLS = [700, 1003, 131072, 300000]


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _close_or_infinite(got, want, bound):
    """close(), where a value beyond f32's range is its infinity."""
    with np.errstate(over="ignore"):
        out = np.isinf(want.astype(np.float32))
    g = got.detach().double().cpu().numpy()
    assert np.array_equal(g[out], np.sign(want[out]) * np.inf), (g[out], want[out])
    inside = torch.from_numpy(~out).to(got.device)
    close(got[inside], want[~out], bound[~out], "f32")


def _check(R, x, xv, t, scale, gt, kl=0.0, modes=("logp", "value", "gradient")):
    """Every call over these rows against the oracle; old_logp leaves ratios of 1, or of 0 where logp is so
    far down that its own rounding would decide the ratio."""
    rows, cols = xv.shape
    logp = OT.token_logp(xv, t, scale)[0]
    old = np.where(logp < -1e4, -3.0, logp).astype(np.float32)
    adv = np.where(np.arange(rows) % 2 == 0, 1.5, -0.75).astype(np.float32)
    w = np.linspace(0.2, 0.9, rows).astype(np.float32)
    ref = (old + np.float32(0.25)) if kl else None
    want = OT.policy_loss(xv, t, old, ref, adv, w, 0.2, 0.25, kl, scale)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    targets = dev(t)
    if "logp" in modes:
        out = torch.full((rows,), float("nan"), device="cuda")
        R.psk_token_logp(x, targets, out, scale=scale)
        value, bound, _, _ = OT.token_logp(xv, t, scale)
        _close_or_infinite(out, value, bound)
    ws = scratch(R.psk_policy_loss_workspace(rows, cols))
    for mode in modes:
        if mode == "logp":
            continue
        loss, out = torch.full((2,), float("nan"), device="cuda"), torch.full((rows,), float("nan"), device="cuda")
        d = torch.full((rows, cols), float("nan"), dtype=DT[gt], device="cuda") if mode == "gradient" else None
        R.psk_policy_loss(x, targets, dev(old), dev(adv), dev(w), loss, out, d, ref_logp=dev(ref), clip_low=0.2,
                          clip_high=0.25, kl_coef=kl, scale=scale, workspace=ws)
        torch.cuda.synchronize()
        close(loss, *want["loss"], "f32")
        _close_or_infinite(out, *want["logp"])
        if d is not None:
            # An exponential below 2^-126 is taken as zero, in the fused form one of up to sqrt(2) times as much:
            # with the row's coefficient |a| = |w dterm scale|, the ratio at most 1.25 here, an absolute error
            # below 2^-125 |a| on top of the relative ones.
            flushed = 2.0 ** -125 * 1.25 * np.abs(w * adv)[:, None].astype(np.float64) * scale
            value, bound = want["dlogits"]
            close(d, value, bound + flushed, gt)
    assert R.psk_device_status() == 0


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("lt,gt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("scale", [0.8, 1.0, 1.25])
def test_a_target_at_the_lowest_value(R, cols, lt, gt, scale):
    """A mask's usual fill on the target itself: logp is scale times the lowest value (-inf past f32's
    range), the ratio 0, the row's gradient zero and the call's loss finite."""
    rng = np.random.default_rng(cols)
    a = rng.normal(size=(5, cols)) * 2.5
    t = rng.integers(0, cols, 5)
    low = torch.finfo(DT[lt]).min
    a[0, t[0]] = low
    a[1] = low                                    # the target refused beside one allowed token
    a[1, (t[1] + cols // 2) % cols] = 10.0
    a[3, t[3]] = low                              # with a negative advantage: clipped
    a[4, :], a[4, t[4]] = low, 4.0                # the one allowed token
    x, xv = stored(a, lt)
    _check(R, x, xv, t, scale, gt)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("lt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 0.4, 1.0])
def test_a_difference_beyond_the_range(R, cols, lt, scale):
    """x_t - max passes f32's range; scaled by less than a half its product does not."""
    rng = np.random.default_rng(cols + 1)
    a = rng.normal(size=(4, cols)) * 2.5
    t = rng.integers(0, cols, 4)
    for r in (0, 1, 3):
        a[r, (t[r] + 1 + cols // 3) % cols] = 3e38
    a[0, t[0]], a[1, t[1]], a[3, t[3]] = -3e38, -1e38, -2.5e38
    x, xv = stored(a, lt)
    _check(R, x, xv, t, scale, lt)


def _far_rows(cols, top, step):
    """Six rows whose maximum is `top`, with `step` the distance of neighbouring values there: all equal;
    two levels, the token at the upper and at the lower one; all at -top; a ladder of neighbouring values; one
    far above the others."""
    rng = np.random.default_rng(cols)
    a = np.full((6, cols), top)
    lower = rng.random((2, cols)) < 0.5
    a[1:3][lower] -= 2.0 ** 17 * step
    t = rng.integers(0, cols, 6)
    a[1, t[1]] = a[2, (t[2] + 1) % cols] = top
    a[2, t[2]] = top - 2.0 ** 17 * step
    a[3] = -top
    a[4] -= step * rng.integers(0, 16, cols)
    a[4, t[4]] = top
    a[5] = rng.normal(size=cols) * top / 64
    a[5, t[5]] = top
    return a, t


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("lt", ["bf16", "f32"])
@pytest.mark.parametrize("through", ["logits", "scale"])
@pytest.mark.parametrize("power", [20, 23, 24, 27, 29, 31, 34, 60, 99])
def test_scaled_logits_far_from_zero(R, cols, lt, through, power):
    """scale * max from 2^20 to 2^99 (1.37 times it: no power of two, whose products would be exact)."""
    far = 1.37 * 2.0 ** power
    top, scale = (far, 1.0) if through == "logits" else (10.0, far / 10.0)
    a, t = _far_rows(cols, top, 2.0 ** (np.floor(np.log2(top)) - 23))
    x, xv = stored(a, lt)
    _check(R, x, xv, t, scale, lt)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("lt", ["bf16", "f32"])
def test_tiny_logits_at_the_largest_scale(R, cols, lt):
    a, t = _far_rows(cols, 5e-22, 2.0 ** -94)       # scale * max = 5e8; a gradient of 1e29
    x, xv = stored(a, lt)
    _check(R, x, xv, t, 1e30, lt)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("lt", ["bf16", "f32"])
def test_nearly_certain_tokens(R, cols, lt):
    """The target's probability within 2^-8 to 2^-30 of one, the runner-up beside it, in another 16-byte group
    or half a row away: the other entries keep their digits, the target's carries the absolute error of logp."""
    places = (1, 17, cols // 2)
    a = np.full((12, cols), -104.0)
    t = (np.arange(12) * 53) % cols
    for r in range(12):
        a[r, t[r]] = 0.0
        a[r, (t[r] + places[r % 3]) % cols] = np.log(2.0) * -(8, 16, 25, 30)[r // 3]
    x, xv = stored(a, lt)
    _check(R, x, xv, t, 1.0, lt, kl=0.1)
