"""Refusals of the training operators (embedding, dropout, norm backward,
token log-probabilities, policy loss) on the host: nothing is launched, so no
GPU is needed and the addresses are made up."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

A, B, C, D, E, F_, G, H, W = (0x10000000 * k for k in range(1, 10))   # far apart
F32, BF16, I32, I64 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def native():
    from reduction_groups_gb300 import build as BD

    BD.build()
    from reduction_groups_gb300 import _native as N

    return N


def _refused(native, rc, name, text=""):
    assert native.ERRORS.get(rc) == name, (rc, native.lib().psk_last_error())
    assert text in native.lib().psk_last_error().decode()


EMBED = dict(ids=A, idt=I64, tokens=4, table=B, tt=BF16, vocab=10, cols=8, ldt=8, scale=1.0, y=C, yt=BF16, ldy=8, s=0)


@pytest.mark.parametrize("change,name", [
    (dict(idt=F32), "PSK_E_DTYPE"), (dict(tt=I32), "PSK_E_DTYPE"), (dict(yt=7), "PSK_E_DTYPE"),
    (dict(tokens=-1), "PSK_E_SHAPE"), (dict(vocab=1 << 31), "PSK_E_SHAPE"), (dict(ldt=7), "PSK_E_SHAPE"),
    (dict(ldy=7), "PSK_E_SHAPE"), (dict(ldy=1 << 60), "PSK_E_SHAPE"), (dict(ids=0), "PSK_E_NULL"),
    (dict(table=0), "PSK_E_NULL"), (dict(y=0), "PSK_E_NULL"), (dict(ids=A + 4), "PSK_E_ARG"),
    (dict(scale=float("nan")), "PSK_E_ARG"), (dict(scale=float("inf")), "PSK_E_ARG"),
    (dict(y=B + 16), "PSK_E_ALIAS"), (dict(y=A), "PSK_E_ALIAS"),
])
def test_embed_refusals(native, change, name):
    _refused(native, native.lib().psk_embed(*{**EMBED, **change}.values()), name)


def test_empty_calls_launch_nothing(native):
    L = native.lib()
    assert L.psk_embed(*{**EMBED, "tokens": 0, "ids": 0, "y": 0}.values()) == 0
    assert L.psk_embed_backward(0, I64, 0, 0, F32, 8, 1.0, B, F32, 10, 8, 8, 1, 0, 0, 0) == 0   # accumulate nothing
    assert L.psk_dropout(0, F32, 0, 0, 0, F32, 0, 8, 8, 0, 8, 0.5, 1, 0, 0, 0) == 0
    assert L.psk_norm_backward(0, F32, 0, F32, 0, F32, 0, 8, 8, 8, 8, 0, 1e-6, 0, 0, 0, 0, 0, 0, 0, 0) == 0
    assert L.psk_token_logp(0, F32, 0, 8, 8, 1.0, 0, I64, 0, 0) == 0


def _embed_ws(native, tokens=4, vocab=10, cols=8):
    v = ctypes.c_uint64(0)
    assert native.lib().psk_embed_workspace(tokens, vocab, cols, ctypes.byref(v)) == 0
    return v.value


@pytest.mark.parametrize("change,name", [
    (dict(idt=BF16), "PSK_E_DTYPE"), (dict(ct_t=I64), "PSK_E_DTYPE"), (dict(dt=I32), "PSK_E_DTYPE"),
    (dict(cols=-2), "PSK_E_SHAPE"), (dict(ldc=7), "PSK_E_SHAPE"), (dict(ldd=7), "PSK_E_SHAPE"),
    (dict(ids=0), "PSK_E_NULL"), (dict(ct=0), "PSK_E_NULL"), (dict(d=0), "PSK_E_NULL"), (dict(ws=0), "PSK_E_NULL"),
    (dict(ws=W + 8), "PSK_E_ARG"), (dict(wb=-1), "PSK_E_ARG"), (dict(scale=float("inf")), "PSK_E_ARG"),
    (dict(d=B), "PSK_E_ALIAS"), (dict(d=A - 16), "PSK_E_ALIAS"), (dict(d=W), "PSK_E_ALIAS"),
    (dict(ws=B), "PSK_E_ALIAS"), (dict(ws=A), "PSK_E_ALIAS"),
])
def test_embed_backward_refusals(native, change, name):
    ok = dict(ids=A, idt=I64, tokens=4, ct=B, ct_t=F32, ldc=8, scale=1.0, d=C, dt=F32, vocab=10, cols=8, ldd=8,
              accumulate=0, ws=W, wb=_embed_ws(native), s=0)
    if change.get("wb") == -1:
        change = dict(wb=ok["wb"] - 1)
    _refused(native, native.lib().psk_embed_backward(*{**ok, **change}.values()), name)


@pytest.mark.parametrize("change,name", [
    (dict(xt=I32), "PSK_E_DTYPE"), (dict(rt=I64), "PSK_E_DTYPE"), (dict(yt=-1), "PSK_E_DTYPE"),
    (dict(p=1.5), "PSK_E_ARG"), (dict(p=-0.1), "PSK_E_ARG"), (dict(p=float("nan")), "PSK_E_ARG"),
    (dict(rows=-1), "PSK_E_SHAPE"), (dict(cols=(1 << 34) + 1, ldx=1 << 35, ldy=1 << 35), "PSK_E_SHAPE"),
    (dict(ldx=7), "PSK_E_SHAPE"), (dict(ldr=7), "PSK_E_SHAPE"), (dict(ldy=1 << 60), "PSK_E_SHAPE"),
    (dict(x=0), "PSK_E_NULL"), (dict(y=0), "PSK_E_NULL"), (dict(counter=D + 4), "PSK_E_ARG"),
    (dict(y=A + 32), "PSK_E_ALIAS"), (dict(y=A, yt=BF16), "PSK_E_ALIAS"), (dict(y=B, ldy=9), "PSK_E_ALIAS"),
    (dict(counter=C + 8), "PSK_E_ALIAS"),
])
def test_dropout_refusals(native, change, name):
    ok = dict(x=A, xt=F32, res=B, rt=F32, y=C, yt=F32, rows=4, cols=8, ldx=8, ldr=8, ldy=8, p=0.5, seed=1, offset=2,
              counter=0, s=0)
    _refused(native, native.lib().psk_dropout(*{**ok, **change}.values()), name)


def _norm_ws(native, rows=4, cols=8):
    v = ctypes.c_uint64(0)
    assert native.lib().psk_norm_backward_workspace(rows, cols, ctypes.byref(v)) == 0
    return v.value


@pytest.mark.parametrize("change,name", [
    (dict(xt=I32), "PSK_E_DTYPE"), (dict(ct_t=9), "PSK_E_DTYPE"), (dict(dxt=I64), "PSK_E_DTYPE"),
    (dict(pt=I32), "PSK_E_DTYPE"), (dict(gt=I32), "PSK_E_DTYPE"), (dict(kind=2), "PSK_E_ARG"),
    (dict(eps=float("inf")), "PSK_E_ARG"), (dict(kind=0), "PSK_E_ARG"), (dict(cols=49153), "PSK_E_SHAPE"),
    (dict(rows=-1), "PSK_E_SHAPE"), (dict(ldc=7), "PSK_E_SHAPE"), (dict(x=0), "PSK_E_NULL"), (dict(ct=0), "PSK_E_NULL"),
    (dict(dx=0), "PSK_E_NULL"), (dict(ws=0), "PSK_E_NULL"), (dict(ws=W + 4), "PSK_E_ARG"), (dict(wb=-1), "PSK_E_ARG"),
    (dict(dx=A + 32), "PSK_E_ALIAS"), (dict(dx=B, dxt=BF16), "PSK_E_ALIAS"), (dict(dx=D), "PSK_E_ALIAS"),
    (dict(dg=F_), "PSK_E_ALIAS"), (dict(dg=D), "PSK_E_ALIAS"), (dict(dg=C), "PSK_E_ALIAS"), (dict(db=W), "PSK_E_ALIAS"),
    (dict(ws=A), "PSK_E_ALIAS"), (dict(ws=D), "PSK_E_ALIAS"),
])
def test_norm_backward_refusals(native, change, name):
    ok = dict(x=A, xt=F32, ct=B, ct_t=F32, dx=C, dxt=F32, rows=4, cols=8, ldx=8, ldc=8, ldd=8, kind=1, eps=1e-5,
              gamma=D, pt=F32, dg=E, db=F_, gt=F32, ws=W, wb=_norm_ws(native), s=0)
    if change.get("wb") == -1:
        change = dict(wb=ok["wb"] - 1)
    _refused(native, native.lib().psk_norm_backward(*{**ok, **change}.values()), name)


@pytest.mark.parametrize("change,name", [
    (dict(lt=I32), "PSK_E_DTYPE"), (dict(tt=F32), "PSK_E_DTYPE"), (dict(cols=0), "PSK_E_SHAPE"),
    (dict(ldl=7), "PSK_E_SHAPE"), (dict(scale=0.0), "PSK_E_ARG"), (dict(scale=-1.0), "PSK_E_ARG"),
    (dict(scale=float("inf")), "PSK_E_ARG"), (dict(x=0), "PSK_E_NULL"), (dict(t=0), "PSK_E_NULL"),
    (dict(logp=0), "PSK_E_NULL"), (dict(t=B + 4), "PSK_E_ARG"), (dict(logp=C + 2), "PSK_E_ARG"),
    (dict(logp=A), "PSK_E_ALIAS"), (dict(logp=B), "PSK_E_ALIAS"),
])
def test_token_logp_refusals(native, change, name):
    ok = dict(x=A, lt=F32, rows=4, cols=8, ldl=8, scale=1.0, t=B, tt=I64, logp=C, s=0)
    _refused(native, native.lib().psk_token_logp(*{**ok, **change}.values()), name)


@pytest.mark.parametrize("change,name", [
    (dict(lt=I64), "PSK_E_DTYPE"), (dict(tt=BF16), "PSK_E_DTYPE"), (dict(gt=I32), "PSK_E_DTYPE"),
    (dict(rows=-1), "PSK_E_SHAPE"), (dict(ldl=7), "PSK_E_SHAPE"), (dict(ldg=7), "PSK_E_SHAPE"),
    (dict(lo=1.5), "PSK_E_ARG"), (dict(hi=-0.1), "PSK_E_ARG"), (dict(kl=float("nan")), "PSK_E_ARG"),
    (dict(old=D + 1), "PSK_E_ARG"), (dict(old=0), "PSK_E_NULL"), (dict(adv=0), "PSK_E_NULL"), (dict(ref=0), "PSK_E_NULL"),
    (dict(loss=0), "PSK_E_NULL"), (dict(ws=0), "PSK_E_NULL"), (dict(ws=W + 8), "PSK_E_ARG"), (dict(wb=15), "PSK_E_ARG"),
    (dict(g=A, gt=BF16), "PSK_E_ALIAS"), (dict(g=A + 32), "PSK_E_ALIAS"), (dict(g=B), "PSK_E_ALIAS"),
    (dict(loss=C), "PSK_E_ALIAS"), (dict(logp=A), "PSK_E_ALIAS"), (dict(logp=H), "PSK_E_ALIAS"),
    (dict(ws=G), "PSK_E_ALIAS"), (dict(ws=E), "PSK_E_ALIAS"), (dict(ws=A), "PSK_E_ALIAS"),
])
def test_policy_loss_refusals(native, change, name):
    ok = dict(x=A, lt=F32, rows=4, cols=8, ldl=8, scale=1.0, t=B, tt=I64, old=C, ref=D, adv=E, weight=F_, lo=0.2,
              hi=0.2, kl=0.1, loss=H, logp=H + 4096, g=G, gt=F32, ldg=8, ws=W, wb=1 << 20, s=0)
    _refused(native, native.lib().psk_policy_loss(*{**ok, **change}.values()), name)


def test_embed_backward_refuses_rows_too_far_apart(native):
    L, far = native.lib(), (1 << 29) + 8
    ok = dict(ids=A, idt=I64, tokens=4, ct=B, ct_t=F32, ldc=8, scale=1.0, d=C, dt=F32, vocab=10, cols=8, ldd=8,
              accumulate=0, ws=W, wb=_embed_ws(native), s=0)
    for change in (dict(ldc=far), dict(ldd=far)):
        _refused(native, L.psk_embed_backward(*{**ok, **change}.values()), "PSK_E_SHAPE")


def test_workspace_sizes(native):
    L, v = native.lib(), ctypes.c_uint64(0)
    assert _embed_ws(native, 0, 10, 8) == 0 and _embed_ws(native, 1, 1, 1) > 0
    assert _embed_ws(native, 1 << 20, 32000, 2048) < (1 << 20) * 2048 * 4 // 8
    assert _norm_ws(native, 0, 8) == 0
    assert L.psk_policy_loss_workspace(-1, 8, ctypes.byref(v)) < 0
    for f, args in ((L.psk_embed_workspace, (1, 1, 1)), (L.psk_norm_backward_workspace, (1, 1)),
                    (L.psk_policy_loss_workspace, (1, 1))):
        _refused(native, f(*args, None), "PSK_E_NULL")


def test_binding_refuses_what_it_cannot_pass_on(native):
    import reduction_groups_gb300 as R

    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA device"):
        R.psk_dropout(x, torch.zeros(4, 8), 0.5, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        R.psk_embed(torch.zeros(4, dtype=torch.int64), x, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="one device"):
        R.psk_token_logp(x, torch.zeros(4, dtype=torch.int64, device="meta"), torch.zeros(4))


def test_binding_torch_is_complete_before_it_shows(monkeypatch):
    """A call on another thread binds for itself until every lookup is bound: whatever torch attribute the
    binding reads, the flag that calls go by must not be set yet."""
    import sys
    import types

    from reduction_groups_gb300 import ops

    for name in ("_F32", "_current_device", "_current_stream"):
        monkeypatch.setattr(ops, name, None)
    read = []

    class Watched(types.ModuleType):
        def __init__(self, real):
            super().__init__("torch")
            self.__dict__["_real"] = real

        def __getattr__(self, name):
            read.append(name)
            assert ops._F32 is None or None not in (ops._current_device, ops._current_stream), name
            v = getattr(self._real, name)
            return Watched(v) if name in ("_C", "cuda") else v

    monkeypatch.setitem(sys.modules, "torch", Watched(torch))
    ops._bind_torch()
    assert "_C" in read and ops._F32 is torch.float32
    assert ops._current_device is not None and ops._current_stream is not None
