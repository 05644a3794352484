"""The head kernels behind a kernel that leaves NaN words in every SM's shared
memory: what a head's own columns do not fill must not reach its results."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_rotary import _check
from tests.train_util import scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


class _Behind:
    """The library, its head operators each behind a product of NaN (its ring of
    operand stages takes nearly all of an SM's shared memory, on every SM)."""

    def __init__(self, R):
        self.R = R
        self.x, self.w = (torch.full(s, float("nan"), device="cuda", dtype=torch.bfloat16) for s in ((8192, 1024), (1024, 2048)))
        self.y = torch.empty(8192, 2048, device="cuda", dtype=torch.bfloat16)
        self.ws = scratch(R.psk_linear_workspace(self.x, self.w))

    def __getattr__(self, name):
        call = getattr(self.R, name)
        if not name.startswith("psk_qk_norm_rotary") or name.endswith("workspace"):
            return call

        def behind(*args):
            self.R.psk_linear(self.x, self.w, self.y, workspace=self.ws)
            call(*args)

        return behind


@pytest.mark.parametrize("dim,rot", [(24, 24), (40, 24), (80, 80), (96, 96), (96, 32), (112, 112), (320, 160), (50, 20)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_left_in_shared_memory_is_read(R, dim, rot, pairs, dtype):
    _check(_Behind(R), 300, 5, 2, dim, rot, "rms", pairs, dtype)
