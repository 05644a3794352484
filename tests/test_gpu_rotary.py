"""psk_qk_norm_rotary and its backward against their binary64 definition,
within the bounds of f32 arithmetic and the storage roundings."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.guard import guarded
from tests.train_util import DT, close, scratch, stored

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _inputs(rng, tokens, hq, hk, dim, rot, xt, far, packed):
    if packed:                                        # columns of the qkv product's rows
        qkv, v = stored(1.5 * rng.normal(size=(tokens, (hq + 2 * hk) * dim)), xt)
        qkv, v = qkv.view(tokens, hq + 2 * hk, dim), v.reshape(tokens, hq + 2 * hk, dim)
        q, k, qv, kv = qkv[:, :hq], qkv[:, hq:hq + hk], v[:, :hq], v[:, hq:hq + hk]
    else:
        (q, qv), (k, kv) = (stored(1.5 * rng.normal(size=(tokens, h, dim)), xt) for h in (hq, hk))
    pos = rng.integers(-far, far + 1, tokens) if far else np.arange(tokens)
    freqs = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    return q, k, qv, kv, pos, freqs


def _check(R, tokens, hq, hk, dim, rot, norm="rms", pairs="halves", xt="bf16", yt=None, gt="f32", ct_t=None, dxt=None,
           dgt="f32", far=0, packed=True, inplace=False, pt=torch.int64, seed=0):
    rng = np.random.default_rng(tokens + hq * 3 + hk + dim * 7 + rot + seed)
    yt, ct_t, dxt = yt or xt, ct_t or xt, dxt or xt
    q, k, qv, kv, pos, freqs = _inputs(rng, tokens, hq, hk, dim, rot, xt, far, packed)
    gq, gqv = stored(1 + 0.2 * rng.normal(size=dim), gt) if norm == "rms" and gt else (None, None)
    gk, gkv = stored(1 + 0.2 * rng.normal(size=dim), gt) if norm == "rms" and gt else (None, None)
    p, f = torch.from_numpy(pos).to(pt).cuda(), torch.from_numpy(freqs).cuda()
    ang = OM.angles(pos, freqs)
    # the backward first: the forward may be in place
    (cq, cqv), (ck, ckv) = (stored(rng.normal(size=(tokens, h, dim)), ct_t) for h in (hq, hk))
    gdq, gdk = guarded((tokens, hq, dim), DT[dxt]), guarded((tokens, hk, dim), DT[dxt])
    dgq, dgk = guarded((dim,), DT[dgt]), guarded((dim,), DT[dgt])
    dq, dk = (cq, ck) if inplace else (gdq.tensor, gdk.tensor)
    sums = norm == "rms"
    R.psk_qk_norm_rotary_backward(cq, ck, q, k, dq, dk, p, f, gq, gk, dgq.tensor if sums else None,
                                  dgk.tensor if sums else None, norm, EPS, pairs,
                                  scratch(R.psk_qk_norm_rotary_backward_workspace(tokens, hq, hk, dim)))
    gy = guarded((tokens, hq, dim), DT[yt]), guarded((tokens, hk, dim), DT[yt])
    yq, yk = (q, k) if inplace else (gy[0].tensor, gy[1].tensor)
    R.psk_qk_norm_rotary(q, k, yq, yk, p, f, gq, gk, norm, EPS, pairs)
    torch.cuda.synchronize()
    assert all(g.intact() for g in (gdq, gdk, dgq, dgk) + gy)
    for x, y, ct, dx, dg, g in ((qv, yq, cqv, dq, dgq, gqv), (kv, yk, ckv, dk, dgk, gkv)):
        close(y, *OM.head_norm_turn(x, ang, g, EPS, norm, pairs), yt)
        (wx, ex), wg = OM.head_norm_turn_backward(ct, x, ang, g, EPS, norm, pairs)
        close(dx, wx, ex, dxt)
        if sums:
            close(dg.tensor, *wg, dgt)
        else:
            assert bool(dg.tensor.isnan().all())


SHAPES = [(1, 1, 1, 1, 0), (1, 2, 1, 2, 2), (40, 8, 2, 64, 64), (33, 6, 6, 50, 20), (17, 3, 1, 128, 64), (5, 4, 4, 80, 80),
          (9, 2, 2, 33, 32), (3, 1, 1, 512, 512), (3, 5, 1, 511, 2), (70, 32, 4, 96, 96), (7, 3, 2, 256, 0), (6, 1, 9, 40, 24),
          (300, 4, 4, 128, 128), (4, 17, 3, 16, 16), (5, 2, 2, 144, 32), (3, 2, 2, 200, 130), (2, 3, 3, 320, 160)]


@pytest.mark.parametrize("tokens,hq,hk,dim,rot", SHAPES)
@pytest.mark.parametrize("norm,pairs", [("rms", "halves"), ("rms", "neighbours"), ("none", "halves"), ("none", "neighbours")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_binary64(R, tokens, hq, hk, dim, rot, norm, pairs, dtype):
    _check(R, tokens, hq, hk, dim, rot, norm, pairs, dtype)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (50, 20), (128, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_far_positions(R, pairs, dim, rot, dtype):
    _check(R, 40, 6, 2, dim, rot, "rms", pairs, dtype, far=1 << 40, inplace=True)
    _check(R, 40, 6, 2, dim, rot, "none", pairs, dtype, far=1 << 30, inplace=True, packed=False, pt=torch.int32)


@pytest.mark.parametrize("xt,yt,gt,ct_t,dxt,dgt", [("bf16", "f32", "bf16", "f32", "bf16", "bf16"),
                                                   ("f32", "bf16", None, "bf16", "f32", "f32"),
                                                   ("bf16", "bf16", "f32", "bf16", "f32", "f32"),
                                                   ("f32", "f32", "bf16", "f32", "bf16", "f32")])
@pytest.mark.parametrize("dim,rot", [(64, 64), (50, 30)])
def test_mixed_types(R, xt, yt, gt, ct_t, dxt, dgt, dim, rot):
    _check(R, 60, 5, 3, dim, rot, "rms", "halves", xt, yt, gt, ct_t, dxt, dgt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens(R, dtype):
    _check(R, 5000, 4, 1, 64, 64, "rms", "halves", dtype)
    _check(R, 3001, 3, 2, 50, 50, "rms", "neighbours", dtype)


def test_queries_or_keys_alone(R):
    rng = np.random.default_rng(1)
    q, k, qv, kv, pos, freqs = _inputs(rng, 30, 4, 2, 64, 64, "bf16", 0, True)
    p, f = torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda()
    both = torch.empty(30, 4, 64, device="cuda"), torch.empty(30, 2, 64, device="cuda")
    R.psk_qk_norm_rotary(q, k, *both, p, f)
    for i, x in enumerate((q, k)):
        y = torch.empty_like(both[i])
        R.psk_qk_norm_rotary(*((x, None, y, None) if i == 0 else (None, x, None, y)), p, f)
        assert torch.equal(y, both[i])
        ct, dx, dg = torch.randn_like(y), torch.empty_like(y), torch.empty(64, device="cuda")
        ws = scratch(R.psk_qk_norm_rotary_backward_workspace(30, x.shape[1] if i == 0 else 0, x.shape[1] if i else 0, 64))
        two = lambda t: (t, None) if i == 0 else (None, t)  # noqa: E731
        R.psk_qk_norm_rotary_backward(*two(ct), *two(x), *two(dx), p, f, None, None, *two(dg), workspace=ws)
        (wx, ex), wg = OM.head_norm_turn_backward(ct.cpu().numpy(), (qv, kv)[i], OM.angles(pos, freqs), None, EPS, "rms",
                                                  "halves")
        close(dx, wx, ex, "f32")
        close(dg, *wg, "f32")


@pytest.mark.parametrize("dim,rot", [(64, 64), (50, 20)])
def test_head_after_head(R, dim, rot):
    x, c = (torch.randn(40, 5, dim, device="cuda") for _ in range(2))
    p, f = torch.arange(40, device="cuda"), torch.logspace(0, -3, rot // 2, device="cuda")
    y, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty(dim, device="cuda")
    ws = scratch(R.psk_qk_norm_rotary_backward_workspace(40, 5, 0, dim))
    R.psk_qk_norm_rotary(x, None, y, None, p, f)
    R.psk_qk_norm_rotary_backward(c, None, x, None, dx, None, p, f, None, None, dg, None, workspace=ws)
    turned = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    x2, c2, y2, dx2, dg2 = turned(x), turned(c), turned(y), turned(dx), torch.empty_like(dg)
    y2.zero_(), dx2.zero_()
    R.psk_qk_norm_rotary(x2, None, y2, None, p, f)
    R.psk_qk_norm_rotary_backward(c2, None, x2, None, dx2, None, p, f, None, None, dg2, None, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_no_tokens_give_zero_scale_gradients(R):
    e = torch.empty(0, 3, 64, device="cuda")
    p, f = torch.empty(0, device="cuda", dtype=torch.int64), torch.empty(0, device="cuda")
    dg = [torch.full((64,), float("nan"), device="cuda") for _ in range(2)]
    R.psk_qk_norm_rotary(e, e, e, e, p, f)
    R.psk_qk_norm_rotary_backward(e, e, e, e, e, e, p, f, None, None, *dg,
                                  workspace=scratch(R.psk_qk_norm_rotary_backward_workspace(0, 3, 3, 64)))
    assert not bool(dg[0].any()) and not bool(dg[1].any())


def test_zero_nan_and_infinite_heads_stay_alone(R):
    x = torch.randn(6, 4, 64, device="cuda")
    p, f = torch.arange(6, device="cuda"), torch.logspace(0, -3, 32, device="cuda")
    clean, y = torch.empty_like(x), torch.empty_like(x)
    R.psk_qk_norm_rotary(x, None, clean, None, p, f)
    x[0, 0], x[2, 1, 5], x[4, 3, 60] = 0.0, float("nan"), float("inf")
    R.psk_qk_norm_rotary(x, None, y, None, p, f)
    assert not bool(y[0, 0].any()) and bool(y[2, 1].isnan().all())
    other = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    other[0, 0] = other[2, 1] = other[4, 3] = False
    assert torch.equal(y[other], clean[other])
    f[3] = float("nan")                              # a frequency that is not a number shows in its pair
    R.psk_qk_norm_rotary(x, None, y, None, p, f)
    assert bool(y[1, :, [3, 35]].isnan().all()) and bool(y[1, :, 4:35].isfinite().all())


def test_rows_beside_the_heads_are_left_alone(R):
    buf = torch.full((20, 9, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    buf[:, 1:4], buf[:, 5:6] = torch.randn(20, 3, 64, device="cuda").bfloat16(), torch.randn(20, 1, 64, device="cuda").bfloat16()
    p, f = torch.arange(20, device="cuda"), torch.logspace(0, -3, 32, device="cuda")
    R.psk_qk_norm_rotary(buf[:12, 1:4], buf[:12, 5:6], buf[:12, 1:4], buf[:12, 5:6], p[:12].clone(), f)
    for h in (0, 4, 6, 7, 8):
        assert bool((buf[:, h] == 7.0).all())
    assert bool(buf[:12, 1:4].isfinite().all())


def test_repeats_bit_for_bit_on_a_side_stream_and_in_a_graph(R):
    x, c = torch.randn(700, 6, 64, device="cuda"), torch.randn(700, 6, 64, device="cuda")
    p, f = torch.arange(700, device="cuda"), torch.logspace(0, -3, 32, device="cuda")
    outs = [(torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda"),
             scratch(R.psk_qk_norm_rotary_backward_workspace(700, 6, 0, 64))) for _ in range(3)]

    def run(o, stream=None):
        R.psk_qk_norm_rotary(x, None, o[0], None, p, f, stream=stream)
        R.psk_qk_norm_rotary_backward(c, None, x, None, o[1], None, p, f, None, None, o[2], None, workspace=o[3],
                                      stream=stream)

    run(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(outs[1], side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[2])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0][:3], o[:3]))


@pytest.mark.parametrize("dim", [64, 50])
def test_no_turning_columns_need_no_positions(R, dim):
    import reduction_groups_gb300._native as N

    x, y, dx = (torch.randn(9, 3, dim, device="cuda") for _ in range(3))
    want, wdx = torch.empty_like(x), torch.empty_like(x)
    p, f = torch.arange(9, device="cuda"), torch.empty(0, device="cuda")
    R.psk_qk_norm_rotary(x, None, want, None, p, f)
    R.psk_qk_norm_rotary_backward(x, None, x, None, wdx, None, p, f)
    s = torch.cuda.current_stream().cuda_stream
    head = lambda t: (t.data_ptr(), None, N.PSK_F32, 3 * dim, dim, 0, 0)  # noqa: E731
    rest = (9, 3, 0, dim, 0, None, N.PSK_I64, None, N.PSK_PAIRS_HALVES, N.PSK_HEAD_NORM_RMS, 1e-6, None, None, 0)
    N.check(N.lib().psk_qk_norm_rotary(*head(x), *head(y), *rest, s))
    N.check(N.lib().psk_qk_norm_rotary_backward(*head(x), *head(x), *head(dx), *rest, None, None, 0, None, 0, s))
    assert torch.equal(y, want) and torch.equal(dx, wdx)
