"""psk_embed and psk_embed_backward against the oracle: the lookup bit for bit
(one product), the gradient bit for bit in its declared order and within the
binary64 bound."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.training as OT
from tests.guard import guarded
from tests.train_util import DT, close, same_bits, scratch, stored, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


def _ids(rng, n, vocab, it, kind="mixed"):
    if kind == "one":
        a = np.full(n, vocab // 2)
    elif kind == "none":
        a = np.full(n, -1)
    else:
        a = (np.exp(rng.uniform(0, np.log(vocab + 1), n)) - 1).astype(np.int64)
        a[rng.random(n) < 0.05] = -1
        a[rng.random(n) < 0.02] = vocab          # past the table: padding as well
        if it == "i64":
            a[rng.random(n) < 0.02] = (1 << 40) + 1
    return a, torch.from_numpy(a.astype(np.int64 if it == "i64" else np.int32)).cuda()


@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (1, 92, 64), (7, 92, 65), (33, 1000, 8), (257, 511, 771),
                                               (64, 32000, 2048), (5, 3, 4104)])
@pytest.mark.parametrize("tt,yt,it", [("f32", "f32", "i32"), ("bf16", "bf16", "i64"), ("bf16", "f32", "i32"),
                                      ("f32", "bf16", "i64")])
def test_lookup_bitwise(R, tokens, vocab, cols, tt, yt, it):
    rng = np.random.default_rng(tokens * 31 + cols)
    a, ids = _ids(rng, tokens, vocab, it)
    table, tv = stored(rng.normal(size=(vocab, cols)), tt)
    g = guarded((tokens, cols), DT[yt])
    R.psk_embed(ids, table, g.tensor, scale=cols ** 0.5)
    torch.cuda.synchronize()
    assert g.intact()
    same_bits(g.tensor, OT.embed(a, tv, cols ** 0.5), yt)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (1, 0)])
def test_lookup_strided_rows(R, pad, offset):
    rng = np.random.default_rng(8)
    a, ids = _ids(rng, 90, 50, "i64")
    table, tv = stored(rng.normal(size=(50, 72)), "bf16")
    y = torch.full((90, 72 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    R.psk_embed(ids, strided(table, pad, offset), y[:, :72])
    same_bits(y[:, :72].contiguous(), OT.embed(a, tv, 1.0), "bf16")
    assert bool((y[:, 72:] == 7.0).all())


GRADS = [(1, 1, 1, "mixed"), (1, 92, 64, "mixed"), (31, 92, 65, "mixed"), (32, 5, 8, "one"), (33, 5, 9, "one"),
         (64, 40, 256, "mixed"), (65, 3, 771, "mixed"), (2000, 92, 64, "mixed"), (1000, 7, 2048, "mixed"),
         (40, 70000, 24, "mixed"), (515, 300, 40, "none"), (4096, 9, 16, "one"), (9000, 300, 16, "mixed"),
         (40000, 70000, 8, "mixed"), (70001, 11, 3, "mixed")]


@pytest.mark.parametrize("tokens,vocab,cols,kind", GRADS)
@pytest.mark.parametrize("ct_t,dt,it", [("f32", "f32", "i32"), ("bf16", "bf16", "i64"), ("bf16", "f32", "i64")])
def test_gradient_bitwise_in_declared_order(R, tokens, vocab, cols, kind, ct_t, dt, it):
    rng = np.random.default_rng(tokens + cols)
    a, ids = _ids(rng, tokens, vocab, it, kind)
    ct, cv = stored(rng.normal(size=(tokens, cols)), ct_t)
    g = guarded((vocab, cols), DT[dt])
    ws = scratch(R.psk_embed_workspace(tokens, vocab, cols))
    R.psk_embed_backward(ids, ct, g.tensor, scale=1.7, workspace=ws)
    torch.cuda.synchronize()
    assert g.intact()
    want, _ = OT.embed_backward_f32(a, cv, vocab, 1.7)
    same_bits(g.tensor, want, dt)
    # and against binary64: n additions of terms of the sum of magnitudes, the scale's and product's rounding
    n = np.bincount(a[(a >= 0) & (a < vocab)].astype(np.int64), minlength=vocab)[:, None]
    close(g.tensor, OT.embed_backward(a, cv, vocab, 1.7),
          (n + 3) * OT.U * OT.embed_backward(a, np.abs(cv), vocab, 1.7), dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (5, 1)])
def test_gradient_accumulates_into_the_rows_that_occur(R, dt, pad, offset):
    rng = np.random.default_rng(6)
    a, ids = _ids(rng, 700, 400, "i64")
    ct, cv = stored(rng.normal(size=(700, 136)), "bf16")
    old, ov = stored(rng.normal(size=(400, 136)), dt)
    d = strided(old, pad, offset)
    ws = scratch(R.psk_embed_workspace(700, 400, 136))
    R.psk_embed_backward(ids, strided(ct, pad, offset), d, scale=0.5, accumulate=True, workspace=ws)
    g, seen = OT.embed_backward_f32(a, cv, 400, 0.5)
    same_bits(d.contiguous(), np.where(seen[:, None], ov + g, ov), dt)
    assert not seen.all()


def test_gradient_of_no_tokens_is_zero(R):
    d = torch.full((300, 17), float("nan"), device="cuda")
    R.psk_embed_backward(torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 17, device="cuda"), d)
    assert not bool(d.any())


def test_padding_rows_of_the_cotangent_are_not_read_into_sums(R):
    ids = torch.tensor([3, -1, 3, 9, 4, 3], device="cuda")
    ct = torch.ones(6, 40, device="cuda")
    ct[1], ct[3] = float("nan"), float("inf")           # positions -1 and 9 (a vocabulary of 9)
    d = torch.empty(9, 40, device="cuda")
    R.psk_embed_backward(ids, ct, d, workspace=scratch(R.psk_embed_workspace(6, 9, 40)))
    want = torch.zeros(9, 40)
    want[3], want[4] = 3.0, 1.0
    assert torch.equal(d.cpu(), want)


def test_side_stream_and_captured_replays(R):
    rng = np.random.default_rng(9)
    vocab, cols, tokens = 500, 96, 800
    ws = scratch(R.psk_embed_workspace(tokens, vocab, cols))
    table, tv = stored(rng.normal(size=(vocab, cols)), "bf16")
    ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    ct = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    y, d = torch.empty_like(ct), torch.empty(vocab, cols, dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    R.psk_embed(ids, table, y, stream=side)
    R.psk_embed_backward(ids, ct, d, workspace=ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.psk_embed(ids, table, y)
        R.psk_embed_backward(ids, ct, d, workspace=ws)
    for _ in range(3):
        a, new = _ids(rng, tokens, vocab, "i64")
        c, cv = stored(rng.normal(size=(tokens, cols)), "bf16")
        ids.copy_(new)
        ct.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        same_bits(y, OT.embed(a, tv, 1.0), "bf16")
        same_bits(d, OT.embed_backward_f32(a, cv, vocab, 1.0)[0], "f32")


@pytest.mark.parametrize("tokens,vocab,cols,kind", [(128, 5, 264, "one"), (128, 3, 40, "mixed"), (127, 200, 33, "mixed"),
                                                    (100, 2, 512, "mixed"), (129, 4, 24, "mixed"), (128, 9, 8, "none")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_short_lists(R, tokens, vocab, cols, kind, accumulate):
    rng = np.random.default_rng(tokens * 5 + vocab)
    a, ids = _ids(rng, tokens, vocab, "i64", kind)
    ct, cv = stored(rng.normal(size=(tokens, cols)), "bf16")
    d, dv = stored(rng.normal(size=(vocab, cols)), "f32")
    R.psk_embed_backward(ids, ct, d, scale=0.7, accumulate=accumulate,
                         workspace=scratch(R.psk_embed_workspace(tokens, vocab, cols)))
    g, seen = OT.embed_backward_f32(a, cv, vocab, 0.7)
    same_bits(d, np.where(seen[:, None], dv + g, dv) if accumulate else g, "f32")


def test_a_large_table_of_few_tokens(R):
    rng = np.random.default_rng(12)
    for tokens in (3, 300):
        a, ids = _ids(rng, tokens, 400000, "i32")
        ct, cv = stored(rng.normal(size=(tokens, 24)), "f32")
        d = torch.full((400000, 24), float("nan"), device="cuda")
        R.psk_embed_backward(ids, ct, d, workspace=scratch(R.psk_embed_workspace(tokens, 400000, 24)))
        same_bits(d, OT.embed_backward_f32(a, cv, 400000, 1.0)[0], "f32")
