"""Calls at once: expert FFNs, products and choices on two streams from two
threads, and two graphs replayed side by side, on shared weights and inputs with
scratch of their own: the bits of the calls one after another."""
from concurrent.futures import ThreadPoolExecutor

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()
    yield
    assert A.afd_mx4_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK


def layer(counts, hidden, inter, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    E, n = len(counts), sum(counts)

    def packed(M, K, swiglu):
        q = R.mx4_quantize(torch.randn(E * M, K, generator=g, device="cuda") / K ** 0.5)
        return R.Mx4Weight(q.codes.view(E, M, -1), q.scales.view(E, M, -1), swiglu=swiglu)

    x = torch.randn(n, hidden, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    logits = torch.randn(n, 64, generator=g, device="cuda")
    return x, off, packed(2 * inter, hidden, True), packed(hidden, inter, False), logits


def work(x, off, w13, wd, logits):
    q = R.mx4_quantize(x)
    ids, w = R.route_select(logits, 6, renorm=True)
    return R.mx4_ffn(q, off, w13, wd), R.mx4_gemm(q, off, w13), R.mx4_gemm(q, off, w13), ids, w


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


# few rows a group and many, so that narrow and wide kernels meet
@pytest.mark.parametrize("counts", [([20] * 32, [500, 0, 900, 333]), ([700, 800], [600, 1000]), ([3] * 16, [9] * 16)])
def test_two_threads_two_streams(counts):
    layers = [layer(c, 512, 352, i) for i, c in enumerate(counts)]
    want = [work(*l) for l in layers]
    torch.cuda.synchronize()

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [work(*layers[(i + j) % 2]) for j in range(30)]
        stream.synchronize()
        return A.afd_mx4_poll_status(stream.cuda_stream), all(same(r, want[(i + j) % 2]) for j, r in enumerate(got))

    with ThreadPoolExecutor(2) as ex:
        assert list(ex.map(run, range(2))) == [(A.AFD_OK, True)] * 2


def test_two_graphs_side_by_side():
    layers = [layer(c, 512, 352, i) for i, c in enumerate(([20] * 32, [500, 0, 900, 333]))]
    want = [work(*l) for l in layers]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for l in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([work(*l) for _ in range(5)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(same(r, w) for r in o)
