"""silu far below zero: its values until they leave f32's normal range."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.train_util import DT, scratch

pytestmark = pytest.mark.gpu


def _silu(z):
    return z / (1.0 + np.exp(-z))


@pytest.mark.parametrize("dtype,half", [("f32", 2.0 ** -20), ("bf16", 2.0 ** -8 + 2.0 ** -16)])
@pytest.mark.parametrize("rows", [3, 700])
def test_silu_keeps_its_tail(dtype, half, rows):
    """z is the bias alone (zero operands): -130 to -60 and beside them ordinary values.  f32: the function's 2^-20;
    bf16: half a step and the coarser form's 2^-16.  Below 2^-126 within steps of 2^-149 (bf16: 2^-133)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    z = torch.linspace(-130.0, -60.0, 1024, device="cuda").to(DT[dtype])
    z[::7] = torch.linspace(-20.0, 20.0, len(z[::7]), device="cuda").to(DT[dtype])
    x, w = torch.zeros(rows, 64, device="cuda", dtype=DT[dtype]), torch.zeros(64, 1024, device="cuda", dtype=DT[dtype])
    y = torch.empty(rows, 1024, device="cuda", dtype=DT[dtype])
    R.psk_linear(x, w, y, z, "silu", workspace=scratch(R.psk_linear_workspace(x, w)))
    want = _silu(z.double().cpu().numpy())
    step = 2.0 ** -148 if dtype == "f32" else 2.0 ** -133
    assert (np.abs(y.double().cpu().numpy() - want) <= half * np.abs(want) + step).all()
