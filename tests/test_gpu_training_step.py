"""The training operators as one step uses them: embedding, dropout, the norm
region, a linear head (torch), the policy loss with its gradient, the norm's,
dropout's and embedding's backward, and AdamW on the resulting leaves --
against the same step in binary64 with torch's automatic differentiation."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.adamw as OA
import oracle.training as OT
from synth.workloads import AdamWHyper
from tests.train_util import scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("captured", [False, True])
def test_step_gradients_and_update(R, kind, captured):
    V, D, T = 92, 64, 96
    p, seed, offset, eps, kl = 0.1, 77, 5, 1e-5, 0.05
    rng = np.random.default_rng(10)
    f32 = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda()  # noqa: E731
    table, head, gamma, beta = f32(V, D), f32(D, V) / 8, 1 + 0.1 * f32(D), 0.1 * f32(D)
    ids = torch.from_numpy(rng.integers(-1, V, T)).cuda()
    targets = torch.from_numpy(rng.integers(0, V, T)).cuda()
    adv, w = f32(T), torch.full((T,), 1.0 / T, device="cuda")
    w[:9] = 0.0
    keep = torch.from_numpy(OT.dropout_keep(T, D, p, seed, offset)).cuda()

    # the step in binary64
    leaves = [t.double().requires_grad_() for t in (table, gamma, beta)]
    tab, ga, be = leaves
    h = torch.where((ids >= 0)[:, None], tab[ids.clamp(min=0)] * 2.0, 0.0) * keep * float(np.float32(1 / (1 - p)))
    c = h - h.mean(1, keepdim=True) if kind == "layer" else h
    n = c / (c.square().mean(1, keepdim=True) + float(np.float32(eps))).sqrt() * ga
    n = n + be if kind == "layer" else n
    logp = torch.log_softmax(n @ head.double(), 1).gather(1, targets[:, None])[:, 0]
    # sampled under weights some updates behind: ratios away from the bounds
    old = (logp.detach() - torch.from_numpy(np.log(rng.choice([0.6, 0.9, 1.1, 1.5], T))).cuda()).float()
    ref = (logp.detach() + 0.3 * f32(T)).float()
    r, q = (logp - old.double()).exp(), ref.double() - logp
    loss = (w.double() * (-torch.minimum(r * adv.double(), r.clamp(0.8, 1.2) * adv.double())
                          + kl * (q.expm1() - q))).sum()
    loss.backward()

    # the step through the library
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    h0, h1, h2, logits, gl = e(T, D), e(T, D), e(T, D), e(T, V), e(2)
    dn, dh1, dh0, dt, dg, db = e(T, D), e(T, D), e(T, D), e(V, D), e(D), e(D)
    ws = [scratch(R.psk_policy_loss_workspace(T, V)), scratch(R.psk_norm_backward_workspace(T, D)),
          scratch(R.psk_embed_workspace(T, V, D))]
    m, v = [torch.zeros_like(t) for t in (table, gamma, beta)], [torch.zeros_like(t) for t in (table, gamma, beta)]
    start = [t.clone() for t in (table, gamma, beta)]
    hp = AdamWHyper(t=1)
    head_t = head.t().contiguous()

    def step():
        R.psk_embed(ids, table, h0, scale=2.0)
        R.psk_dropout(h0, h1, p, seed, offset)
        R.psk_norm_region(h1, h2, kind, eps, gamma, beta if kind == "layer" else None)
        torch.mm(h2, head, out=logits)
        R.psk_policy_loss(logits, targets, old, adv, w, gl, None, logits, ref_logp=ref, kl_coef=kl, workspace=ws[0])
        torch.mm(logits, head_t, out=dn)
        R.psk_norm_backward(h1, dn, dh1, kind, eps, gamma, dg, db if kind == "layer" else None, ws[1])
        R.psk_dropout(dh1, dh0, p, seed, offset)
        R.psk_embed_backward(ids, dh0, dt, scale=2.0, workspace=ws[2])
        tree = [(table, m[0], v[0], dt), (gamma, m[1], v[1], dg)] + ([(beta, m[2], v[2], db)] if kind == "layer" else [])
        R.psk_adamw_tree(tree, hp)

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                   # warm-up: the matrix products' handles
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, s in zip((table, gamma, beta), start):
            t.copy_(s)
        for t in m + v:
            t.zero_()
        graph.replay()
    else:
        step()
    torch.cuda.synchronize()

    # f32 through ten operations of depth up to 96: the head's products carry
    # 64 and 92 terms (error below 92 u of the sums of magnitudes, about ten
    # times the sums here), logits of about 8 an absolute error of 8 * 92 u =
    # 4.4e-5 at worst, and the gradients that relative error a few times over.
    want = float(loss.detach())
    assert abs(float(gl[0]) - want) < 2e-4 * (1 + abs(want))
    for got, leaf in zip((dt, dg) + ((db,) if kind == "layer" else ()), leaves):
        want = leaf.grad
        assert float((got.double() - want).norm()) < 5e-4 * float(want.norm())
    # AdamW saw exactly these gradients
    got = OA.step_tree([(start[0].cpu().numpy().ravel(), np.zeros(V * D, np.float32), np.zeros(V * D, np.float32),
                         dt.cpu().numpy().ravel())], "f32", hp)[0]
    assert np.array_equal(table.cpu().numpy().ravel().view(np.uint32), got[0].view(np.uint32))
    assert R.psk_device_status() == 0
