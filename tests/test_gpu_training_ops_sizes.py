"""The training operators at training sizes, bit for bit: the kernels' variants
that only large calls take (several groups of columns a thread, eight columns
a lane of the run sums, a table zeroed partly beside the sort)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.training as OT
from tests.guard import guarded
from tests.train_util import DT, same_bits, scratch, stored, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


# Four groups a thread (rows x padded row / 32 of at least 2048 an SM), whole
# spans and a ragged last one; two, likewise.
@pytest.mark.parametrize("rows,cols", [(4096, 4096), (2700, 4056), (3300, 1536), (3400, 1520)])
@pytest.mark.parametrize("xt,rt,yt", [("bf16", "bf16", "bf16"), ("bf16", None, "bf16"), ("f32", "f32", "f32"),
                                      ("bf16", "f32", "f32"), ("f32", None, "bf16")])
def test_dropout(R, rows, cols, xt, rt, yt):
    rng = np.random.default_rng(rows + cols)
    x, xv = stored(rng.standard_normal((rows, cols), dtype=np.float32), xt)
    r, rv = stored(rng.standard_normal((rows, cols), dtype=np.float32), rt) if rt else (None, None)
    g = guarded((rows, cols), DT[yt])
    R.psk_dropout(x, g.tensor, 0.1, 77, 1 << 33, residual=r)
    torch.cuda.synchronize()
    assert g.intact()
    want = OT.dropout(xv, rv, 0.1, 77, 1 << 33)
    same_bits(g.tensor, want, yt)
    if xt == yt:
        R.psk_dropout(x, x, 0.1, 77, 1 << 33, residual=r)
        same_bits(x, want, yt)


@pytest.mark.parametrize("cols", [4096, 4056])
def test_dropout_of_rows_in_wider_buffers(R, cols):
    rng = np.random.default_rng(cols)
    x, xv = stored(rng.standard_normal((2700, cols), dtype=np.float32), "bf16")
    r, rv = stored(rng.standard_normal((2700, cols), dtype=np.float32), "bf16")
    buf = torch.full((2700, cols + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    R.psk_dropout(strided(x, 8), buf[:, 8:8 + cols], 0.3, 5, residual=strided(r, 16))
    same_bits(buf[:, 8:8 + cols].contiguous(), OT.dropout(xv, rv, 0.3, 5, 0), "bf16")
    assert bool((buf[:, :8] == 7.0).all()) and bool((buf[:, 8 + cols:] == 7.0).all())


def _ids(rng, n, vocab):
    """Ids falling as 1 / rank, padding before and past the table among them."""
    a = np.minimum((np.exp(rng.uniform(0, np.log(vocab + 1), n)) - 1).astype(np.int64), vocab - 1)
    a = rng.permutation(vocab)[a]
    a[rng.random(n) < 0.03] = -1
    a[rng.random(n) < 0.02] = vocab
    return a, torch.from_numpy(a).cuda()


# Four groups a lane: bf16 tables of 1024 columns and more, 32 warps an SM.
@pytest.mark.parametrize("tokens,cols", [(5000, 1032), (5000, 1033), (2500, 2048), (1700, 3001)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_lookup(R, tokens, cols, yt):
    rng = np.random.default_rng(tokens + cols)
    a, ids = _ids(rng, tokens, 700)
    table, tv = stored(rng.standard_normal((700, cols), dtype=np.float32), "bf16")
    g = guarded((tokens, cols), DT[yt])
    R.psk_embed(ids, table, g.tensor, scale=cols ** 0.5)
    torch.cuda.synchronize()
    assert g.intact()
    same_bits(g.tensor, OT.embed(a, tv, cols ** 0.5), yt)


# Eight columns a lane (16 run slices an SM); of a CTA's slice of the table the
# first rows are zeroed beside the sort, the others looked up; all of them; and
# rows that begin anywhere, none of them.
@pytest.mark.parametrize("tokens,vocab,cols", [(16384, 32000, 2048), (20000, 50000, 1024), (40000, 9000, 512),
                                               (12000, 20000, 2049)])
@pytest.mark.parametrize("ct_t,dt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_gradient(R, tokens, vocab, cols, ct_t, dt):
    rng = np.random.default_rng(tokens + cols)
    a, ids = _ids(rng, tokens, vocab)
    ct, cv = stored(rng.standard_normal((tokens, cols), dtype=np.float32), ct_t)
    g = guarded((vocab, cols), DT[dt])
    R.psk_embed_backward(ids, ct, g.tensor, scale=1.7, workspace=scratch(R.psk_embed_workspace(tokens, vocab, cols)))
    torch.cuda.synchronize()
    assert g.intact()
    want, seen = OT.embed_backward_f32(a, cv, vocab, 1.7)
    assert 0 < int(seen.sum()) < vocab
    same_bits(g.tensor, want, dt)


# The same sizes added to a leaf (four columns a lane).
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_added_to_a_leaf(R, dt):
    rng = np.random.default_rng(4)
    a, ids = _ids(rng, 16384, 32000)
    ct, cv = stored(rng.standard_normal((16384, 1024), dtype=np.float32), "bf16")
    d, dv = stored(rng.standard_normal((32000, 1024), dtype=np.float32), dt)
    R.psk_embed_backward(ids, ct, d, scale=0.5, accumulate=True, workspace=scratch(R.psk_embed_workspace(16384, 32000, 1024)))
    g, seen = OT.embed_backward_f32(a, cv, 32000, 0.5)
    same_bits(d, np.where(seen[:, None], dv + g, dv), dt)
