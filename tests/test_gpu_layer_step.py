"""The matrix operators as one layer's step uses them: the norm region, the
qkv product, the norm and rotation of its heads in place, attention (torch),
the output product added to the residual stream, a feed-forward pair, all
their backwards, and the orthogonalised update of the matrices -- against the
same layer in binary64 with torch's automatic differentiation."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.train_util import scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _attend(q, k, v):
    """Causal attention of [T, heads, D], a key head shared by hq / hk query heads."""
    T, hq, D = q.shape
    k, v = (t.repeat_interleave(hq // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("thd,shd->hts", q, k) / D ** 0.5
    s = s.masked_fill(torch.ones(T, T, device=q.device, dtype=torch.bool).triu(1), float("-inf"))
    return torch.einsum("hts,shd->thd", s.softmax(-1), v).flatten(1)


@pytest.mark.parametrize("captured", [False, True])
def test_layer_gradients_and_update(R, captured):
    T, C, HQ, HK, D, FF = 96, 64, 4, 2, 16, 256
    H = HQ + 2 * HK
    rng = np.random.default_rng(20)
    f32 = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda()  # noqa: E731
    x, ct = f32(T, C), f32(T, C)
    leaves = [1 + 0.1 * f32(C), f32(C, H * D) / 8, 0.1 * f32(H * D), 1 + 0.1 * f32(D), 1 + 0.1 * f32(D), f32(HQ * D, C) / 8,
              f32(C, FF) / 8, 0.1 * f32(FF), f32(FF, C) / 16]
    g0, wqkv, bqkv, gq, gk, wo, w1, b1, w2 = leaves
    pos = torch.arange(T, device="cuda") + 5000
    freqs = torch.from_numpy((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)).cuda()
    eps = 1e-5

    # the layer in binary64
    X = x.double().requires_grad_()
    G0, WQ, BQ, GQ, GK, WO, W1, B1, W2 = L64 = [t.double().requires_grad_() for t in leaves]
    rms = lambda t, g: t / (t.square().mean(-1, keepdim=True) + float(np.float32(eps))).sqrt() * g  # noqa: E731
    qkv = (rms(X, G0) @ WQ + BQ).view(T, H, D)
    ang = torch.from_numpy(OM.angles(pos.cpu().numpy(), freqs.cpu().numpy())).cuda()[:, None]

    def turned(u):
        a, b = u[..., :D // 2], u[..., D // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    h = X + _attend(turned(rms(qkv[:, :HQ], GQ)), turned(rms(qkv[:, HQ:HQ + HK], GK)), qkv[:, HQ + HK:]) @ WO
    y = h + torch.nn.functional.gelu(h @ W1 + B1) @ W2
    want = torch.autograd.grad((y * ct.double()).sum(), [X] + L64)

    # through the library
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    n, qkv, att, h, z1, a1, y = e(T, C), e(T, H, D), e(T, HQ * D), e(T, C), e(T, FF), e(T, FF), e(T, C)
    dx, dn, dqkv, datt, dh, da1, tmp = e(T, C), e(T, C), e(T, H, D), e(T, HQ * D), e(T, C), e(T, FF), e(T, C)
    grads = [torch.empty_like(t) for t in leaves]
    dg0, dwqkv, dbqkv, dgq, dgk, dwo, dw1, db1, dw2 = grads
    updates = [torch.empty_like(t) for t in (wqkv, wo, w1, w2)]
    raw = e(T, H, D)
    flat = lambda t: t.view(T, H * D)  # noqa: E731
    q, k, v = (lambda t: (t[:, :HQ], t[:, HQ:HQ + HK], t[:, HQ + HK:]))(qkv)
    need = max(R.psk_linear_workspace(n, wqkv), R.psk_linear_workspace(h, w1), R.psk_linear_workspace(a1, w2),
               R.psk_linear_workspace(att, wo), R.psk_linear_backward_workspace(ct, a1, w2, da1, dw2),
               R.psk_linear_backward_workspace(da1, h, w1, tmp, dw1, db1, act="gelu"),
               R.psk_linear_backward_workspace(dh, att, wo, datt, dwo),
               R.psk_linear_backward_workspace(flat(dqkv), n, wqkv, dn, dwqkv, dbqkv), R.psk_norm_backward_workspace(T, C),
               R.psk_qk_norm_rotary_backward_workspace(T, HQ, HK, D))
    ws = scratch(need)                                  # one stream: the calls' workspaces in turn
    osizes = [R.psk_orthogonalize_workspace(1, *t.shape, t.dtype) for t in updates]
    ows = scratch(max(osizes))

    def step():
        R.psk_norm_region(x, n, "rms", eps, g0)
        R.psk_linear(n, wqkv, flat(raw), bqkv, workspace=ws)
        qkv.copy_(raw)                                  # the backward reads the heads before their norm
        R.psk_qk_norm_rotary(q, k, q, k, pos, freqs, gq, gk, eps=eps)
        with torch.enable_grad():
            qa, ka, va = (t.detach().clone().requires_grad_() for t in (q, k, v))
            o = _attend(qa, ka, va)
        att.copy_(o.detach())
        R.psk_linear(att, wo, h, residual=x, workspace=ws)
        R.psk_linear(h, w1, a1, b1, "gelu", z=z1, workspace=ws)
        R.psk_linear(a1, w2, y, residual=h, workspace=ws)
        R.psk_linear_backward(ct, a1, w2, da1, dw2, workspace=ws)
        R.psk_linear_backward(da1, h, w1, tmp, dw1, db1, act="gelu", z=z1, workspace=ws)
        torch.add(ct, tmp, out=dh)
        R.psk_linear_backward(dh, att, wo, datt, dwo, workspace=ws)
        dq, dk, dv = torch.autograd.grad(o, (qa, ka, va), datt)
        dqkv[:, HQ + HK:].copy_(dv)
        R.psk_qk_norm_rotary_backward(dq, dk, raw[:, :HQ], raw[:, HQ:HQ + HK], dqkv[:, :HQ], dqkv[:, HQ:HQ + HK], pos, freqs,
                                      gq, gk, dgq, dgk, eps=eps, workspace=ws)
        R.psk_linear_backward(flat(dqkv), n, wqkv, dn, dwqkv, dbqkv, workspace=ws)
        R.psk_norm_backward(x, dn, dx, "rms", eps, g0, dg0, None, ws)
        dx.add_(dh)
        for g, u in zip((dwqkv, dwo, dw1, dw2), updates):
            R.psk_orthogonalize([g], [u], scale=0.2 * max(g.shape) ** 0.5, workspace=ows)

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                      # warm-up: the matrix products' handles
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in grads + updates:
            t.fill_(float("nan"))
        graph.replay()
    else:
        step()
    torch.cuda.synchronize()
    # f32 through eleven operations of sums of up to 256 terms (256 u = 1.5e-5 of their magnitudes, a few times the
    # sums here), the attention's and each backward's relative errors added: a few 1e-4 at worst.
    for got, ref in zip([dx] + grads, want):
        assert float((got.double() - ref).norm()) < 5e-4 * float(ref.norm())
    for g, u in zip((dwqkv, dwo, dw1, dw2), updates):
        gv, co = g.cpu().numpy(), [(3.4445, -4.7750, 2.0315)] * 5
        s = 0.2 * max(g.shape) ** 0.5
        ref = OM.orthogonalize(gv, co, 5, 1e-7, s)
        own = np.linalg.norm(OM.orthogonalize_rounded(gv, co, 5, 1e-7, s, 2) - ref)
        # the roundings' own size twice and 15 products' sums in f32, carried on by at most 4
        assert np.linalg.norm(u.double().cpu().numpy() - ref) < 2 * own + 60 * 40 * 2.0 ** -24 * np.linalg.norm(ref)
    assert R.psk_device_status() == 0
