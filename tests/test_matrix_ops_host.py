"""Refusals of the matrix operators (linear layer, orthogonalised update, head
norm and rotation) on the host: nothing is launched, so no GPU is needed and
the addresses are made up."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

A, B, C, D, E, F_, G, H, W = (0x10000000 * k for k in range(1, 10))   # far apart
F32, BF16, I32, I64 = 0, 1, 2, 3
BIG = 1 << 26


@pytest.fixture(scope="module")
def native():
    from reduction_groups_gb300 import build as BD

    BD.build()
    from reduction_groups_gb300 import _native as N

    return N


def _refused(native, rc, name, text=""):
    assert native.ERRORS.get(rc) == name, (rc, native.lib().psk_last_error())
    assert text in native.lib().psk_last_error().decode()


LINEAR = dict(x=A, xt=F32, ldx=8, w=B, wt=F32, ldw=12, layout=0, rows=4, cin=8, cout=12, bias=C, bt=F32, act=2, res=D, rt=F32,
              ldr=12, z=E, zt=F32, ldz=12, y=F_, yt=F32, ldy=12, ws=W, wb=BIG, s=0)


@pytest.mark.parametrize("change,name", [
    (dict(xt=I32), "PSK_E_DTYPE"), (dict(wt=7), "PSK_E_DTYPE"), (dict(bt=I64), "PSK_E_DTYPE"), (dict(rt=-1), "PSK_E_DTYPE"),
    (dict(zt=I32), "PSK_E_DTYPE"), (dict(yt=I32), "PSK_E_DTYPE"), (dict(layout=2), "PSK_E_ARG"), (dict(act=4), "PSK_E_ARG"),
    (dict(act=-1), "PSK_E_ARG"), (dict(rows=-1), "PSK_E_SHAPE"), (dict(rows=1 << 31), "PSK_E_SHAPE"),
    (dict(cin=(1 << 25) + 1, ldx=1 << 26), "PSK_E_SHAPE"), (dict(cout=-1), "PSK_E_SHAPE"), (dict(ldx=7), "PSK_E_SHAPE"),
    (dict(ldw=11), "PSK_E_SHAPE"), (dict(layout=1, ldw=7), "PSK_E_SHAPE"), (dict(ldr=11), "PSK_E_SHAPE"),
    (dict(ldz=11), "PSK_E_SHAPE"), (dict(ldy=11), "PSK_E_SHAPE"), (dict(ldy=1 << 60), "PSK_E_SHAPE"), (dict(x=0), "PSK_E_NULL"),
    (dict(w=0), "PSK_E_NULL"), (dict(y=0), "PSK_E_NULL"), (dict(ws=0), "PSK_E_NULL"), (dict(x=A + 2), "PSK_E_ARG"),
    (dict(bias=C + 1), "PSK_E_ARG"), (dict(y=F_ + 2), "PSK_E_ARG"), (dict(ws=W + 8), "PSK_E_ARG"), (dict(wb=16), "PSK_E_ARG"),
    (dict(y=A), "PSK_E_ALIAS"), (dict(y=B + 16), "PSK_E_ALIAS"), (dict(y=C), "PSK_E_ALIAS"), (dict(y=D + 16), "PSK_E_ALIAS"),
    (dict(y=D, yt=BF16), "PSK_E_ALIAS"), (dict(y=D, ldy=13), "PSK_E_ALIAS"), (dict(y=E), "PSK_E_ALIAS"), (dict(z=A), "PSK_E_ALIAS"),
    (dict(z=D), "PSK_E_ALIAS"), (dict(y=W), "PSK_E_ALIAS"), (dict(z=W), "PSK_E_ALIAS"), (dict(ws=A), "PSK_E_ALIAS"),
    (dict(ws=C), "PSK_E_ALIAS"), (dict(ws=D), "PSK_E_ALIAS"),
])
def test_linear_refusals(native, change, name):
    _refused(native, native.lib().psk_linear(*{**LINEAR, **change}.values()), name)


def test_linear_refuses_columns_of_one_buffer_that_meet(native):
    L = native.lib()
    wide = dict(x=A, ldx=64, y=A + 4 * 7, ldy=64, w=B, res=0, z=0)       # y begins in x's last column
    _refused(native, L.psk_linear(*{**LINEAR, **wide}.values()), "PSK_E_ALIAS", "y overlaps x")
    wide["y"] = A + 4 * 60                                                # y's rows run into x's next row
    _refused(native, L.psk_linear(*{**LINEAR, **wide}.values()), "PSK_E_ALIAS", "y overlaps x")
    wide |= dict(y=A + 4 * 8, wb=16)                                      # side by side: only the workspace is short
    _refused(native, L.psk_linear(*{**LINEAR, **wide}.values()), "PSK_E_ARG", "workspace")


BACK = dict(ct=A, ct_t=F32, ldc=12, x=B, xt=F32, ldx=8, w=C, wt=F32, ldw=12, layout=0, rows=4, cin=8, cout=12, act=2, z=D, zt=F32,
            ldz=12, dx=E, dxt=F32, lddx=8, dw=F_, dwt=F32, lddw=12, db=G, dbt=F32, acc=0, ws=W, wb=BIG, s=0)


@pytest.mark.parametrize("change,name", [
    (dict(ct_t=I32), "PSK_E_DTYPE"), (dict(xt=I64), "PSK_E_DTYPE"), (dict(wt=9), "PSK_E_DTYPE"), (dict(zt=I32), "PSK_E_DTYPE"),
    (dict(dxt=I32), "PSK_E_DTYPE"), (dict(dwt=I32), "PSK_E_DTYPE"), (dict(dbt=I32), "PSK_E_DTYPE"), (dict(layout=-1), "PSK_E_ARG"),
    (dict(act=9), "PSK_E_ARG"), (dict(rows=(1 << 25) + 1), "PSK_E_SHAPE"), (dict(cout=(1 << 25) + 1, ldc=1 << 26), "PSK_E_SHAPE"),
    (dict(cin=-1), "PSK_E_SHAPE"), (dict(ldc=11), "PSK_E_SHAPE"), (dict(ldx=7), "PSK_E_SHAPE"), (dict(ldw=11), "PSK_E_SHAPE"),
    (dict(lddx=7), "PSK_E_SHAPE"), (dict(lddw=11), "PSK_E_SHAPE"), (dict(ldz=11), "PSK_E_SHAPE"), (dict(ct=0), "PSK_E_NULL"),
    (dict(x=0), "PSK_E_NULL"), (dict(w=0), "PSK_E_NULL"), (dict(z=0), "PSK_E_NULL"), (dict(ws=0), "PSK_E_NULL"),
    (dict(ws=W + 4), "PSK_E_ARG"), (dict(wb=16), "PSK_E_ARG"), (dict(dx=E + 1), "PSK_E_ARG"), (dict(dx=A), "PSK_E_ALIAS"),
    (dict(dx=B), "PSK_E_ALIAS"), (dict(dx=C), "PSK_E_ALIAS"), (dict(dx=D), "PSK_E_ALIAS"), (dict(dw=B), "PSK_E_ALIAS"),
    (dict(dw=C), "PSK_E_ALIAS"), (dict(dw=E), "PSK_E_ALIAS"), (dict(db=F_), "PSK_E_ALIAS"), (dict(db=A), "PSK_E_ALIAS"),
    (dict(db=W), "PSK_E_ALIAS"), (dict(ws=B), "PSK_E_ALIAS"), (dict(ws=D), "PSK_E_ALIAS"),
])
def test_linear_backward_refusals(native, change, name):
    _refused(native, native.lib().psk_linear_backward(*{**BACK, **change}.values()), name)


def test_linear_workspaces(native):
    L, v = native.lib(), ctypes.c_uint64(7)
    args = dict(x=A, xt=BF16, ldx=64, w=B, wt=BF16, ldw=96, layout=0, rows=4, cin=64, cout=96)
    size = lambda **c: (L.psk_linear_workspace(*{**args, **c}.values(), ctypes.byref(v)), v.value)  # noqa: E731
    assert size() == (0, 0)
    assert size(ldx=65)[1] > 0 and size(x=A + 2)[1] > 0 and size(xt=F32)[1] >= 3 * 4 * 64 * 2
    assert size(rows=0, xt=F32) == (0, 0)
    _refused(native, L.psk_linear_workspace(*args.values(), None), "PSK_E_NULL")
    _refused(native, size(rows=-1)[0], "PSK_E_SHAPE")
    back = {k: BACK[k] for k in ("ct", "ct_t", "ldc", "x", "xt", "ldx", "w", "wt", "ldw", "layout", "rows", "cin", "cout", "act", "dx",
                                 "dxt", "dw", "dwt", "db", "dbt")}
    assert L.psk_linear_backward_workspace(*back.values(), ctypes.byref(v)) == 0
    whole = v.value
    assert L.psk_linear_backward_workspace(*{**back, "dw": 0}.values(), ctypes.byref(v)) == 0 and v.value < whole
    _refused(native, L.psk_linear_backward_workspace(*back.values(), None), "PSK_E_NULL")


def _ortho(native, n=2, rows=4, cols=8, xt=F32, yt=F32, co=(1.0, 2.0, 3.0), steps=1, eps=1e-7, scale=1.0, ws=W, wb=BIG, ldx=8, ldy=8,
           xs=(A, B), ys=(C, D)):
    leaves = (native.psk_ortho_leaf * 2)()
    for f, x, y in zip(leaves, xs, ys):
        f.x, f.ldx, f.y, f.ldy = x, ldx, y, ldy
    c = (ctypes.c_double * max(1, len(co)))(*co) if co is not None else None
    return native.lib().psk_orthogonalize(leaves, n, rows, cols, xt, yt, c, steps, eps, scale, ws, wb, 0)


@pytest.mark.parametrize("change,name", [
    (dict(n=-1), "PSK_E_ARG"), (dict(n=513), "PSK_E_ARG"), (dict(rows=-1), "PSK_E_SHAPE"), (dict(cols=(1 << 20) + 1), "PSK_E_SHAPE"),
    (dict(xt=I32), "PSK_E_DTYPE"), (dict(yt=I64), "PSK_E_DTYPE"), (dict(steps=0), "PSK_E_ARG"), (dict(steps=65), "PSK_E_ARG"),
    (dict(co=None), "PSK_E_NULL"), (dict(co=(1.0, float("nan"), 1.0)), "PSK_E_ARG"), (dict(co=(33.0, 1.0, 1.0)), "PSK_E_ARG"),
    (dict(eps=-1.0), "PSK_E_ARG"), (dict(eps=float("nan")), "PSK_E_ARG"), (dict(scale=float("inf")), "PSK_E_ARG"),
    (dict(ws=0), "PSK_E_NULL"), (dict(ws=W + 8), "PSK_E_ARG"), (dict(wb=64), "PSK_E_ARG"), (dict(ldx=7), "PSK_E_SHAPE"),
    (dict(ldy=7), "PSK_E_SHAPE"), (dict(ldy=1 << 60), "PSK_E_SHAPE"), (dict(xs=(A, 0)), "PSK_E_NULL"), (dict(ys=(0, D)), "PSK_E_NULL"),
    (dict(xs=(A + 2, B)), "PSK_E_ARG"), (dict(ys=(C, C)), "PSK_E_ALIAS"), (dict(ys=(C, C - 16)), "PSK_E_ALIAS"),
    (dict(xs=(A, W)), "PSK_E_ALIAS"), (dict(ys=(W + 64, D)), "PSK_E_ALIAS"),
])
def test_orthogonalize_refusals(native, change, name):
    _refused(native, _ortho(native, **change), name)


def test_orthogonalize_workspace_and_empty_calls(native):
    L, v = native.lib(), ctypes.c_uint64(0)
    assert L.psk_orthogonalize_workspace(3, 64, 192, BF16, ctypes.byref(v)) == 0
    half = v.value
    assert L.psk_orthogonalize_workspace(3, 64, 192, F32, ctypes.byref(v)) == 0 and v.value > half
    for n, rows, cols in ((0, 5, 5), (1, 0, 5), (1, 5, 0)):
        assert L.psk_orthogonalize_workspace(n, rows, cols, F32, ctypes.byref(v)) == 0 and v.value == 0
        assert _ortho(native, n=n, rows=rows, cols=cols, ws=0, wb=0) == 0
    _refused(native, L.psk_orthogonalize_workspace(1, 5, 5, I32, ctypes.byref(v)), "PSK_E_DTYPE")
    _refused(native, L.psk_orthogonalize_workspace(1, 5, 5, F32, None), "PSK_E_NULL")


ROT = dict(q=A, k=B, xt=F32, qt=32, qh=8, kt=16, kh=8, yq=C, yk=D, yt=F32, yqt=32, yqh=8, ykt=16, ykh=8, tokens=5, hq=4, hk=2, dim=8,
           rot=6, pos=E, pt=I64, freqs=F_, pairs=0, norm=1, eps=1e-6, gq=G, gk=G + 4096, gt=F32, s=0)


@pytest.mark.parametrize("change,name", [
    (dict(xt=I32), "PSK_E_DTYPE"), (dict(yt=5), "PSK_E_DTYPE"), (dict(pt=F32), "PSK_E_DTYPE"), (dict(gt=I32), "PSK_E_DTYPE"),
    (dict(tokens=-1), "PSK_E_SHAPE"), (dict(hq=-1), "PSK_E_SHAPE"), (dict(dim=0, rot=0), "PSK_E_SHAPE"), (dict(dim=513), "PSK_E_SHAPE"),
    (dict(rot=5), "PSK_E_SHAPE"), (dict(rot=10), "PSK_E_SHAPE"), (dict(qh=7), "PSK_E_SHAPE"), (dict(qt=31), "PSK_E_SHAPE"),
    (dict(ykt=15), "PSK_E_SHAPE"), (dict(yqt=1 << 60), "PSK_E_SHAPE"), (dict(pairs=2), "PSK_E_ARG"), (dict(norm=2), "PSK_E_ARG"),
    (dict(eps=-1.0), "PSK_E_ARG"), (dict(eps=float("nan")), "PSK_E_ARG"), (dict(norm=0), "PSK_E_ARG"), (dict(q=0), "PSK_E_NULL"),
    (dict(yk=0), "PSK_E_NULL"), (dict(pos=0), "PSK_E_NULL"), (dict(freqs=0), "PSK_E_NULL"), (dict(q=A + 2), "PSK_E_ARG"),
    (dict(pos=E + 4), "PSK_E_ARG"), (dict(gq=G + 2), "PSK_E_ARG"), (dict(yq=A + 16), "PSK_E_ALIAS"), (dict(yq=A, yqt=40), "PSK_E_ALIAS"),
    (dict(yq=B), "PSK_E_ALIAS"), (dict(yk=A), "PSK_E_ALIAS"), (dict(yk=C), "PSK_E_ALIAS"), (dict(yq=E), "PSK_E_ALIAS"),
    (dict(yq=G), "PSK_E_ALIAS"), (dict(yk=F_), "PSK_E_ALIAS"),
])
def test_rotary_refusals(native, change, name):
    _refused(native, native.lib().psk_qk_norm_rotary(*{**ROT, **change}.values()), name)


ROTB = dict(cq=A, ck=B, ct=F32, cqt=32, cqh=8, ckt=16, ckh=8, q=C, k=D, xt=F32, qt=32, qh=8, kt=16, kh=8, dq=E, dk=F_, dt=F32, dqt=32,
            dqh=8, dkt=16, dkh=8, tokens=5, hq=4, hk=2, dim=8, rot=6, pos=G, pt=I64, freqs=G + 4096, pairs=0, norm=1, eps=1e-6,
            gq=G + 8192, gk=G + 12288, gt=F32, dgq=H, dgk=H + 4096, dgt=F32, ws=W, wb=BIG, s=0)


@pytest.mark.parametrize("change,name", [
    (dict(ct=I32), "PSK_E_DTYPE"), (dict(xt=I32), "PSK_E_DTYPE"), (dict(dt=I32), "PSK_E_DTYPE"), (dict(dgt=I32), "PSK_E_DTYPE"),
    (dict(ckh=7), "PSK_E_SHAPE"), (dict(dqt=31), "PSK_E_SHAPE"), (dict(kt=15), "PSK_E_SHAPE"), (dict(ck=0), "PSK_E_NULL"),
    (dict(k=0), "PSK_E_NULL"), (dict(dq=0), "PSK_E_NULL"), (dict(ws=0), "PSK_E_NULL"), (dict(ws=W + 4), "PSK_E_ARG"),
    (dict(wb=16), "PSK_E_ARG"), (dict(dgq=H + 1), "PSK_E_ARG"), (dict(norm=0, gq=0, gk=0), "PSK_E_ARG"), (dict(dq=B), "PSK_E_ALIAS"),
    (dict(dq=D), "PSK_E_ALIAS"), (dict(dq=A + 16), "PSK_E_ALIAS"), (dict(dk=E), "PSK_E_ALIAS"), (dict(dq=G), "PSK_E_ALIAS"),
    (dict(dgq=A), "PSK_E_ALIAS"), (dict(dgq=H + 4096), "PSK_E_ALIAS"), (dict(dgk=G + 8192), "PSK_E_ALIAS"), (dict(ws=C), "PSK_E_ALIAS"),
    (dict(ws=H), "PSK_E_ALIAS"), (dict(ws=G), "PSK_E_ALIAS"),
])
def test_rotary_backward_refusals(native, change, name):
    _refused(native, native.lib().psk_qk_norm_rotary_backward(*{**ROTB, **change}.values()), name)


def test_rotary_empty_calls(native):
    L, v = native.lib(), ctypes.c_uint64(0)
    none = dict(q=0, k=0, yq=0, yk=0, pos=0, freqs=0)
    assert L.psk_qk_norm_rotary(*{**ROT, **none, "tokens": 0}.values()) == 0
    assert L.psk_qk_norm_rotary(*{**ROT, **none, "hq": 0, "hk": 0, "pos": E, "freqs": F_}.values()) == 0
    back = {**ROTB, "cq": 0, "ck": 0, "q": 0, "k": 0, "dq": 0, "dk": 0, "dgq": 0, "dgk": 0, "ws": 0, "wb": 0, "tokens": 0}
    assert L.psk_qk_norm_rotary_backward(*back.values()) == 0
    assert L.psk_qk_norm_rotary_backward_workspace(100, 4, 2, 64, ctypes.byref(v)) == 0 and v.value > 0
    _refused(native, L.psk_qk_norm_rotary_backward_workspace(100, 4, 2, 64, None), "PSK_E_NULL")
    _refused(native, L.psk_qk_norm_rotary_backward_workspace(100, 4, 2, 0, ctypes.byref(v)), "PSK_E_SHAPE")


def test_binding_refuses_what_it_cannot_pass_on(native):
    import reduction_groups_gb300 as R

    x, w, y = torch.zeros(4, 8), torch.zeros(8, 6), torch.zeros(4, 6)
    with pytest.raises(ValueError, match="CUDA device"):
        R.psk_linear(x, w, y)
    with pytest.raises(ValueError, match="CUDA device"):
        R.psk_orthogonalize([x], [x])
    with pytest.raises(ValueError, match="CUDA device"):
        R.psk_qk_norm_rotary(x[None], None, x[None], None, torch.zeros(1, dtype=torch.int64), torch.zeros(2))
    with pytest.raises(ValueError, match="results"):
        R.psk_orthogonalize([x], [])
    with pytest.raises(ValueError, match="triple"):
        R.psk_orthogonalize([x], [x], steps=2, coefficients=[(1, 2, 3)] * 3)
    with pytest.raises(TypeError, match="storage type"):
        R.psk_orthogonalize_workspace(1, 4, 4, torch.float16)
    assert R.psk_linear_workspace(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 8, dtype=torch.bfloat16)) == 0
    # an [out, in] weight goes in as its transpose, without a copy
    assert R.psk_linear_workspace(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16).t()) == 0
