"""Sums by pieces as programs call them: with the epilogue's inputs, in place,
strided, added to a leaf, lost copies, streams and graphs, host threads."""

import threading

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_linear import _backward, _forward
from tests.train_util import scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import reduction_groups_gb300 as R

    return R


# pairs of CTAs, single ones, few rows, one tile's sum shared
SIZES = [(2100, 2200, 2300), (1500, 2304, 1000), (20, 2500, 20000), (300, 9000, 200)]


@pytest.mark.parametrize("rows,cin,cout", SIZES)
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_epilogue(R, rows, cin, cout, act):
    _forward(R, rows, cin, cout, "bf16", yt="f32", act=act, bias="f32", res="f32", inplace=True)
    _forward(R, rows, cin, cout, "bf16", act=act, bias="bf16", zt="f32", layout="out_in")


@pytest.mark.parametrize("pad", [(8, 0), (3, 1)])
def test_strided(R, pad):
    _forward(R, 700, 2600, 1100, "bf16", yt="f32", act="silu", bias="bf16", res="bf16", pad=pad)
    _backward(R, 2600, 500, 264, "bf16", "none", outs=("f32", "f32"), pad=pad, accumulate=True)


@pytest.mark.parametrize("rows,cin,cout", [(2500, 1500, 1300), (5000, 200, 72), (9000, 64, 40)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_added_to_an_f32_leaf(R, rows, cin, cout, layout):
    _backward(R, rows, cin, cout, "bf16", "none", layout, accumulate=True, outs=("bf16", "f32"))


@pytest.mark.parametrize("rows,cin,cout", SIZES[:3])
@pytest.mark.parametrize("at", [1, 20])
def test_a_lost_copy_ends_in_a_status_not_a_hang(R, rows, cin, cout, at):
    """In the first piece and in a later one."""
    x, w = torch.randn(rows, cin, device="cuda").bfloat16(), torch.randn(cin, cout, device="cuda").bfloat16()
    y, ref = torch.empty(rows, cout, device="cuda"), torch.empty(rows, cout, device="cuda")
    R.psk_linear(x, w, ref, workspace=scratch(R.psk_linear_workspace(x, w)))
    ws = scratch(R.psk_linear_workspace(x, w))
    assert R.psk_device_status(reset=True) == 0
    try:
        R.psk_test_drop_row(at)
        R.psk_linear(x, w, y, workspace=ws)
        torch.cuda.synchronize()
        assert R.psk_device_status(reset=True) == 1
    finally:
        R.psk_test_drop_row(-1)
    R.psk_linear(x, w, y, workspace=ws)
    torch.cuda.synchronize()
    assert R.psk_device_status() == 0 and torch.equal(y, ref)


def _calls(R, seed, size):
    rows, cin, cout = size
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w = torch.randn(rows, cin, generator=g, device="cuda").bfloat16(), torch.randn(cin, cout, generator=g, device="cuda").bfloat16()
    y, dw = torch.empty(rows, cout, device="cuda"), torch.empty(cin, cout, device="cuda")
    ct = torch.randn(rows, cout, generator=g, device="cuda").bfloat16()
    ws = scratch(R.psk_linear_workspace(x, w)), scratch(R.psk_linear_backward_workspace(ct, x, w, None, dw))

    def run(stream=None):
        R.psk_linear(x, w, y, workspace=ws[0], stream=stream)
        R.psk_linear_backward(ct, x, w, None, dw, None, workspace=ws[1], stream=stream)

    return run, (y, dw)


def test_streams_graphs_and_threads_at_once(R):
    sets = [_calls(R, i, s) for i, s in enumerate(SIZES[:2] + [(3000, 300, 257), (260, 4100, 96)])]
    want = []
    for run, out in sets:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for run, _ in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run()

    def by_streams():
        for (run, _), s in zip(sets, streams):
            run(s)

    def by_graphs():
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()

    def by_threads():
        failures = []

        def work(run, s):
            try:
                for _ in range(20):
                    run(s)
            except Exception as e:  # noqa: BLE001
                failures.append(e)

        threads = [threading.Thread(target=work, args=(run, s)) for (run, _), s in zip(sets, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failures

    for call in (by_streams, by_graphs, by_threads):
        for _, out in sets:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        for (_, out), w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w)), call.__name__
    assert R.psk_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_operands_written_on_a_joined_stream_of_a_graph(R, dtype):
    """x is written on a side stream that joins before the call, w on the call's own."""
    d = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x0, w0 = torch.randn(4096, 1024, device="cuda").to(d), torch.randn(1024, 2048, device="cuda").to(d)
    x, w = torch.zeros_like(x0), torch.zeros_like(w0)
    y, ref = torch.empty(4096, 2048, device="cuda"), torch.empty(4096, 2048, device="cuda")
    ws = scratch(R.psk_linear_workspace(x0, w0))
    R.psk_linear(x0, w0, ref, workspace=ws)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                x.add_(1.0)
            x.copy_(x0)
        w.copy_(w0)
        torch.cuda.current_stream().wait_stream(side)
        R.psk_linear(x, w, y, workspace=ws)
    for _ in range(10):
        x.zero_(), w.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
