"""Angles of negative frequencies and of large ones, at far positions."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.matrices as OM
from tests.train_util import close, stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("top", [1.0, 1e3, 1e12])
@pytest.mark.parametrize("dim", [64, 50])
def test_far_angles_of_any_frequency(sign, top, dim):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    rng = np.random.default_rng(dim)
    x, xv = stored(rng.normal(size=(60, 2, dim)), "f32")
    pos = rng.integers(-(1 << 40), 1 << 40, 60)
    freqs = (sign * top * 10000.0 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32)
    y = torch.empty_like(x)
    R.psk_qk_norm_rotary(x, None, y, None, torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda(), norm="none")
    # 2^40 positions of 2^-62 of a turn each: 1.5e-6 radians beside the f32 bound
    want, bound = OM.head_norm_turn(xv, OM.angles(pos, freqs), None, 0.0, "none", "halves")
    close(y, want, bound + 2 * np.pi * 2.0 ** -22 * np.abs(xv).max(), "f32")
