"""Calls of the matrix operators as a program makes them: several streams at
once, one set of parameters in two captured graphs, tensors past 32-bit
offsets, long lists of leaves, the same matrix twice, empty sides."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.train_util import DT, close, scratch, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


class _Layer:
    """One stream's tensors and calls."""

    def __init__(self, R, seed, rows, width, inner, dtype):
        self.R, d = R, DT[dtype]
        torch.manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda").to(d)  # noqa: E731
        self.x, self.w, self.b, self.ct = r(rows, width), r(width, inner) * width ** -0.5, r(inner), r(rows, inner)
        self.p, self.f = torch.arange(rows, device="cuda"), torch.logspace(0, -3, 16, device="cuda")
        self.g = r(32)
        self.upd = [r(width, inner), r(width, inner)]
        e = torch.empty_like
        self.out = [e(self.ct), e(self.ct), e(self.x), e(self.w), e(self.b), e(self.ct), e(self.ct), e(self.g), e(self.upd[0]),
                    e(self.upd[1])]
        y, z, dx, dw, db, q, dq, dg, u, v = self.out
        self.ws = [scratch(R.psk_linear_workspace(self.x, self.w)),
                   scratch(R.psk_linear_backward_workspace(self.ct, self.x, self.w, dx, dw, db, act="silu")),
                   scratch(R.psk_qk_norm_rotary_backward_workspace(rows, inner // 32, 0, 32)),
                   scratch(R.psk_orthogonalize_workspace(2, width, inner, d))]

    def run(self, stream=None):
        R, (y, z, dx, dw, db, q, dq, dg, u, v) = self.R, self.out
        heads = lambda t: t.view(t.shape[0], -1, 32)  # noqa: E731
        R.psk_linear(self.x, self.w, y, self.b, "silu", None, z, self.ws[0], stream)
        R.psk_qk_norm_rotary(heads(y), None, heads(q), None, self.p, self.f, self.g, stream=stream)
        R.psk_qk_norm_rotary_backward(heads(self.ct), None, heads(y), None, heads(dq), None, self.p, self.f, self.g, None, dg,
                                      None, workspace=self.ws[2], stream=stream)
        R.psk_linear_backward(self.ct, self.x, self.w, dx, dw, db, "silu", z, False, self.ws[1], stream)
        R.psk_orthogonalize(self.upd, [u, v], workspace=self.ws[3], stream=stream)


SETS = [[(0, 700, 128, 256, "bf16"), (1, 300, 256, 512, "f32"), (2, 40, 64, 192, "bf16")],
        [(3, 2048, 512, 1024, "bf16"), (4, 2000, 520, 768, "f32"), (5, 2048, 512, 1024, "bf16")]]


@pytest.mark.parametrize("sizes", SETS)
def test_streams_at_once(R, sizes):
    layers = [_Layer(R, *s) for s in sizes]
    want = []
    for m in layers:
        m.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in m.out])
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for m in layers:
            for t in m.out:
                t.zero_()
        torch.cuda.synchronize()
        for m, s in zip(layers, streams):
            m.run(s)
        torch.cuda.synchronize()
        for m, w in zip(layers, want):
            assert all(torch.equal(a, b) for a, b in zip(m.out, w))
    assert R.psk_device_status() == 0


@pytest.mark.parametrize("sizes", SETS)
def test_graphs_at_once(R, sizes):
    """Each set of tensors in a graph of its own; the graphs replayed together, and new inputs seen by each replay."""
    layers = [_Layer(R, *s) for s in sizes]
    graphs, streams = [], [torch.cuda.Stream() for _ in layers]
    for m in layers:
        m.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            m.run()
    for m in layers:
        m.x.mul_(0.5)
        m.upd[1].copy_(m.upd[0])
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for m in layers:
        got = [t.clone() for t in m.out]
        m.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, m.out)) and torch.equal(got[-1], got[-2])


@pytest.mark.parametrize("rows,step", [(40, 1 << 27), (300, 1 << 24)])
def test_offsets_past_32_bits(R, rows, step):
    """Rows far apart: the same results as from packed ones."""
    pool = torch.empty((rows - 1) * step + 4096, device="cuda", dtype=torch.bfloat16)
    far = lambda at, n: pool.as_strided((rows, n), (step, 1), at)  # noqa: E731
    x, w = torch.randn(rows, 320, device="cuda").bfloat16(), (torch.randn(320, 640, device="cuda") / 18).bfloat16()
    ws = scratch(1 << 24)
    y, z = torch.empty(rows, 640, device="cuda", dtype=torch.bfloat16), torch.empty(rows, 640, device="cuda", dtype=torch.bfloat16)
    R.psk_linear(x, w, y, None, "gelu", None, z, ws)
    far(0, 320).copy_(x)
    R.psk_linear(far(0, 320), w, far(320, 640), None, "gelu", None, far(960, 640), ws)
    assert torch.equal(far(320, 640), y) and torch.equal(far(960, 640), z)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(640, device="cuda")
    R.psk_linear_backward(y, x, w, dx, dw, db, "gelu", z, False, ws)
    dw2, db2 = torch.empty_like(w), torch.empty_like(db)
    R.psk_linear_backward(far(320, 640), far(0, 320), w, far(1600, 320), dw2, db2, "gelu", far(960, 640), False, ws)
    assert torch.equal(far(1600, 320), dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    # heads of 64 in both kernels' layouts, and tokens as the far direction
    p, f = torch.arange(rows, device="cuda"), torch.logspace(0, -3, 32, device="cuda")
    for dim, turning in ((64, 32), (80, 10)):
        q, dq = torch.empty(rows, 320 // dim, dim, device="cuda", dtype=torch.bfloat16), torch.empty(rows, 320 // dim, dim, device="cuda", dtype=torch.bfloat16)
        R.psk_qk_norm_rotary(x.view(rows, -1, dim), None, q, None, p, f[:turning].contiguous())
        R.psk_qk_norm_rotary_backward(q, None, x.view(rows, -1, dim), None, dq, None, p, f[:turning].contiguous())
        heads = lambda at: pool.as_strided((rows, 320 // dim, dim), (step, dim, 1), at)  # noqa: E731
        R.psk_qk_norm_rotary(heads(0), None, heads(2048), None, p, f[:turning].contiguous())
        R.psk_qk_norm_rotary_backward(heads(2048), None, heads(0), None, heads(2560), None, p, f[:turning].contiguous())
        assert torch.equal(heads(2048), q) and torch.equal(heads(2560), dq)
    u = torch.empty_like(x)
    R.psk_orthogonalize([x], [u], workspace=ws)
    R.psk_orthogonalize([far(0, 320)], [far(3200, 320)], workspace=ws)
    assert torch.equal(far(3200, 320), u)
    del pool
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,rows,cols", [(40, 24, 48), (512, 8, 16), (33, 130, 300), (512, 20, 260), (3, 1, 700)])
def test_many_leaves(R, n, rows, cols):
    """Every leaf's result is what it gets alone, but for two roundings to bf16 and two of the products' (1e-3 at most)."""
    torch.manual_seed(n)
    xs = [torch.randn(rows, cols, device="cuda") * 1e-3 for _ in range(n)]
    ys, one = [torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(n)], torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    R.psk_orthogonalize(xs, ys, workspace=scratch(R.psk_orthogonalize_workspace(n, rows, cols, torch.bfloat16)))
    ws = scratch(R.psk_orthogonalize_workspace(1, rows, cols, torch.bfloat16))
    for i in sorted({0, 1, n // 2, n - 1}):
        R.psk_orthogonalize([xs[i]], [one], workspace=ws)
        assert float((one.double() - ys[i].double()).norm()) <= 2 * (2.0 ** -8 + 1e-3) * float(one.double().norm())


@pytest.mark.parametrize("rows,cols", [(64, 96), (200, 300)])
def test_one_matrix_in_two_leaves(R, rows, cols):
    x = torch.randn(rows, cols, device="cuda")
    ws = scratch(R.psk_orthogonalize_workspace(2, rows, cols, torch.float32))
    want, other = torch.empty_like(x), torch.empty_like(x)
    R.psk_orthogonalize([x], [want], workspace=ws)
    R.psk_orthogonalize([x, x], [other, x], workspace=ws)          # the second in place
    assert torch.equal(other, want) and torch.equal(x, want)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_sides(R, act, dtype):
    d = DT[dtype]
    e = lambda *s: torch.full(s, 3.0, device="cuda", dtype=d)  # noqa: E731
    # no outputs: dx = 0
    x, w, ct, dx = e(5, 16), e(16, 0), e(5, 0), e(5, 16)
    R.psk_linear_backward(ct, x, w, dx, None, None, act, ct, False, scratch(R.psk_linear_backward_workspace(ct, x, w, dx, act=act)))
    assert not bool(dx.any())
    # no inputs: dbias alone
    x, w, ct, dx, dw, db = e(5, 0), e(0, 8), e(5, 8), e(5, 0), e(0, 8), e(8)
    R.psk_linear_backward(ct, x, w, dx, dw, db, act, e(5, 8), False,
                          scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw, db, act=act)))
    z = torch.full((5, 8), 3.0, device="cuda", dtype=torch.float64, requires_grad=True)
    (torch.nn.functional.gelu(z) if act == "gelu" else z).backward(torch.full((5, 8), 3.0, device="cuda", dtype=torch.float64))
    want = z.grad.sum(0).cpu().numpy()
    close(db, want, np.abs(want) * 2.0 ** -20, dtype)
    # no rows
    y = e(0, 8)
    R.psk_linear(e(0, 16), e(16, 8), y, None, act)


@pytest.mark.parametrize("rows,cin,cout", [(1, 1 << 16, 5), (70000, 3, 2), (2, 5, 70000), (1, 1, 300001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_side_long(R, rows, cin, cout, dtype):
    rng = np.random.default_rng(rows + cin)
    x, xv = stored(rng.normal(size=(rows, cin)), dtype)
    w, wv = stored(rng.normal(size=(cin, cout)) / cin ** 0.5, dtype)
    y = torch.empty(rows, cout, device="cuda", dtype=DT[dtype])
    R.psk_linear(x, w, y, workspace=scratch(R.psk_linear_workspace(x, w)))
    (want, err), _ = OM.linear(xv, wv, None, "none", None, dtype == "f32")
    close(y, want, err, dtype)
    ct, cv = stored(rng.normal(size=(rows, cout)), dtype)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(cout, device="cuda")
    R.psk_linear_backward(ct, x, w, dx, dw, db,
                          workspace=scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw, db)))
    for got, a, b in ((dx, cv, wv.T), (dw, xv.T, cv)):
        (want, err), _ = OM.linear(a, b, None, "none", None, dtype == "f32")
        close(got, want, err, dtype)
    # a column's sum: rows of a warp, eight warps, a quarter of at most 912 blocks one after the other, four quarters
    adds = rows / 7296 + 1 + 8 + min(rows / 32 + 1, 912) / 4 + 1 + 3
    close(db, cv.astype(np.float64).sum(0), np.abs(cv.astype(np.float64)).sum(0) * adds * 2.0 ** -24, "f32")


@pytest.mark.parametrize("n,rows,cols", [(2, 40, 2000), (1, 2100, 60), (3, 300, 3001), (1, 700, 5000), (9, 129, 1800)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_thin_matrices(R, n, rows, cols, yt):
    """Few tiles with a long summed axis: shared out among CTAs."""
    from tests.test_gpu_orthogonalize import _run

    _run(R, n, rows, cols, yt, yt)


@pytest.mark.parametrize("rows,cols,dtype", [(128, 1000, "bf16"), (128, 1000, "f32"), (600, 700, "bf16")])
def test_a_lost_copy_of_the_update_ends_in_a_status(R, rows, cols, dtype):
    x = torch.randn(rows, cols, device="cuda").to(DT[dtype])
    y, ref = torch.empty_like(x), torch.empty_like(x)
    ws = scratch(R.psk_orthogonalize_workspace(1, rows, cols, DT[dtype]))
    R.psk_orthogonalize([x], [ref], 1, workspace=ws)
    assert R.psk_device_status(reset=True) == 0
    try:
        R.psk_test_drop_row(1)
        R.psk_orthogonalize([x], [y], 1, workspace=ws)
        torch.cuda.synchronize()
        assert R.psk_device_status(reset=True) == 1
    finally:
        R.psk_test_drop_row(-1)
    R.psk_orthogonalize([x], [y], 1, workspace=ws)
    torch.cuda.synchronize()
    assert R.psk_device_status() == 0 and torch.equal(y, ref)
