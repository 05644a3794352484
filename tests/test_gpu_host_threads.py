"""Each operator as the first CUDA call that a host thread makes: the same
result as on the main thread."""

import threading

import pytest

torch = pytest.importorskip("torch")

from tests.train_util import scratch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _rand(*shape, dtype=F32):
    return torch.randn(*shape, device="cuda").to(dtype)


def _linear(R, dtype, rows=300):
    x, w, y = _rand(rows, 256, dtype=dtype), _rand(256, 512, dtype=dtype), torch.zeros(rows, 512, device="cuda", dtype=dtype)
    ws = scratch(R.psk_linear_workspace(x, w))
    return lambda s: R.psk_linear(x, w, y, workspace=ws, stream=s), [y]


def _linear_backward(R):
    x, w, ct = _rand(300, 256, dtype=BF16), _rand(256, 512, dtype=BF16), _rand(300, 512, dtype=BF16)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    ws = scratch(R.psk_linear_backward_workspace(ct, x, w, dx, dw))
    return lambda s: R.psk_linear_backward(ct, x, w, dx, dw, workspace=ws, stream=s), [dx, dw]


def _update(R, rows, cols):
    x = _rand(rows, cols, dtype=BF16)
    y = torch.zeros_like(x)
    ws = scratch(R.psk_orthogonalize_workspace(1, rows, cols, BF16))
    return lambda s: R.psk_orthogonalize([x], [y], workspace=ws, stream=s), [y]


def _heads(R):
    x, p, f = _rand(300, 4, 64), torch.arange(300, device="cuda"), torch.logspace(0, -3, 32, device="cuda")
    y, dx, dg = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(64, device="cuda")
    ws = scratch(R.psk_qk_norm_rotary_backward_workspace(300, 4, 0, 64))

    def run(s):
        R.psk_qk_norm_rotary(x, None, y, None, p, f, stream=s)
        R.psk_qk_norm_rotary_backward(x, None, x, None, dx, None, p, f, None, None, dg, workspace=ws, stream=s)

    return run, [y, dx, dg]


def _softmax(R, rows, mode):
    x = _rand(rows, 512, dtype=BF16)
    y = torch.zeros_like(x)
    return lambda s: R.psk_softmax_region(x, y, ("sequential",), mode, stream=s), [y]


def _norm(R, rows):
    x = _rand(rows, 512, dtype=BF16)
    y = torch.zeros_like(x)
    return lambda s: R.psk_norm_region(x, y, "rms", 1e-5, stream=s), [y]


def _embed(R):
    ids, table, y = torch.randint(0, 50, (100,), device="cuda"), _rand(50, 64), torch.zeros(100, 64, device="cuda")
    return lambda s: R.psk_embed(ids, table, y, stream=s), [y]


def _dropout(R):
    x = _rand(100, 64)
    y = torch.zeros_like(x)
    return lambda s: R.psk_dropout(x, y, 0.3, 1, stream=s), [y]


def _logp(R):
    logits, t = _rand(64, 1000, dtype=BF16), torch.randint(0, 1000, (64,), device="cuda")
    y = torch.zeros(64, device="cuda")
    return lambda s: R.psk_token_logp(logits, t, y, stream=s), [y]


def _norm_backward(R):
    x, ct = _rand(100, 512, dtype=BF16), _rand(100, 512, dtype=BF16)
    dx, ws = torch.zeros_like(x), scratch(R.psk_norm_backward_workspace(100, 512))
    return lambda s: R.psk_norm_backward(x, ct, dx, "rms", 1e-5, workspace=ws, stream=s), [dx]


CALLS = {
    "linear bf16": lambda R: _linear(R, BF16), "linear f32": lambda R: _linear(R, F32),
    "linear few rows": lambda R: _linear(R, BF16, 8), "linear backward": _linear_backward,
    "small update": lambda R: _update(R, 64, 128), "update": lambda R: _update(R, 300, 400), "heads": _heads,
    "softmax many rows": lambda R: _softmax(R, 20000, "fast"), "softmax few rows": lambda R: _softmax(R, 100, "fast"),
    "softmax exact": lambda R: _softmax(R, 20000, "exact"), "norm many rows": lambda R: _norm(R, 20000),
    "norm few rows": lambda R: _norm(R, 100), "embed": _embed, "dropout": _dropout, "logp": _logp,
    "norm backward": _norm_backward,
}


@pytest.mark.parametrize("name", CALLS)
def test_a_threads_first_call(R, name):
    run, outs = CALLS[name](R)
    stream = torch.cuda.Stream()
    run(stream)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            run(stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(a, b) for a, b in zip(outs, want))
