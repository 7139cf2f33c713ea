"""afd_route_select against a plain 64-bit choice: ids equal, weights within
the fp32 bound.

A weight's error in units of 2^-24 of itself: the score (softmax: 25 + the
argument's rounding, |l - top| <= 24 here; sigmoid: 6), the sum of 16 and
the division (6), the scaling (1): under 64."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import mx4_reference as ref

W_TOL = 64 * 2.0 ** -24


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def draw(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g, device="cuda")).to(dtype), g


def check(logits, topk, **kw):
    ids, w = R.route_select(logits, topk, **kw)
    rid, rw = ref.select(logits, topk, **kw)
    assert torch.equal(ids.cpu(), rid), (ids.cpu() != rid).any(1).nonzero().flatten()[:5]
    w = w.double().cpu()
    assert torch.equal(torch.isnan(w), torch.isnan(rw))
    fine = ~torch.isnan(rw)
    err = (w[fine] - rw[fine]).abs() - W_TOL * rw[fine].abs()
    assert err.numel() == 0 or float(err.max()) <= 1e-45
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (3, 2, 2), (37, 60, 4), (9, 33, 16), (130, 64, 6),
                                   (65, 100, 3), (64, 128, 8), (33, 129, 7), (70, 255, 5), (66, 256, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_plain(T, E, k, score, dtype):
    logits, g = draw(T, E, 7 * T + E, dtype)
    check(logits, k, score=score)
    check(logits, k, score=score, renorm=True, routed_scaling=2.5)
    check(logits, k, score=score, bias=0.2 * torch.randn(E, generator=g, device="cuda"), renorm=True)


@pytest.mark.parametrize("E,G,tg,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 2, 3), (96, 3, 1, 16), (12, 4, 4, 12),
                                      (30, 2, 1, 15), (32, 32, 5, 5), (250, 5, 2, 9)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, G, tg, k, group_top, score):
    for dtype in (torch.float32, torch.bfloat16):
        logits, g = draw(61, E, E + G, dtype)
        bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        kw = dict(score=score, n_groups=G, topk_groups=tg, group_top=group_top)
        check(logits, k, **kw)
        check(logits, k, bias=bias, renorm=True, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg", [(1, 1), (4, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked(score, G, tg, with_bias):
    """-inf logits and biases: rows with few experts left, one, none."""
    logits, g = draw(200, 48, 3)
    u = torch.rand(200, 48, generator=g, device="cuda")
    logits[u < torch.linspace(0, 1.05, 200, device="cuda").unsqueeze(1)] = -math.inf
    logits[0] = -math.inf
    logits[1, :47] = -math.inf
    logits[1, 47] = 0.25
    bias = None
    if with_bias:
        bias = 0.3 * torch.randn(48, generator=g, device="cuda") - 0.5
        bias[5] = -math.inf
        bias[40] = -math.inf
    ids, w = check(logits, 6, score=score, bias=bias, n_groups=G, topk_groups=tg, group_top=2, renorm=True)
    assert (ids[0] == -1).all() and (w[0] == 0).all()
    assert int(ids[1, 0]) == 47 and (ids[1, 1:] == -1).all() and float(w[1, 0]) == 1.0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg", [(1, 1), (8, 3)])
def test_ties_and_neighbours(score, G, tg):
    """Equal values go to the lower index, values one fp32 step apart to the
    larger: equal rows, bf16 duplicates, zero and equal biases, and scores
    that only fp64 tells apart."""
    E = 64
    base = torch.zeros(4, E, device="cuda")
    base[1, ::3] = 1.0
    base[2] = torch.arange(E, device="cuda") % 5
    base[3] = -0.0
    base[3, ::2] = 0.0
    kw = dict(score=score, n_groups=G, topk_groups=tg, group_top=2)
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.25, device="cuda")):
        check(base, 8, bias=bias, **kw)
    # logits a few fp32 steps apart around 1; biases of the same size
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    steps = torch.randint(0, 40, (500, E), generator=g, device="cuda")
    near = (1.0 + steps * 2.0 ** -23).float()
    bias = torch.randint(0, 3, (E,), generator=g, device="cuda") * 2.0 ** -25
    check(near, 8, bias=bias.float(), **kw)
    if G == 1:
        check(near, 8, **kw)
    coarse, _ = draw(300, E, 5, torch.bfloat16)
    check((coarse * 4).round() / 4, 8, bias=torch.full((E,), 0.125, device="cuda"), **kw)


def test_extremes():
    """Large, tiny and infinite logits, NaN, infinite biases."""
    E = 40
    l, g = draw(64, E, 9, spread=40.0)
    for score in ("softmax", "sigmoid"):
        check(l.clamp(-12, 12), 5, score=score, renorm=True)
    low = torch.full((3, E), -100.0, device="cuda") - torch.arange(E, device="cuda") * 0.5
    ids, w = R.route_select(low, 4, score="sigmoid", renorm=True)
    rid, rw = ref.select(low, 4, score="sigmoid", renorm=True)
    assert torch.equal(ids.cpu(), rid)
    assert (w.double().cpu() / rw - 1).abs().max() < W_TOL
    high = torch.randn(2, E, device="cuda", generator=g)
    high[0, 3] = math.inf
    high[1, 7] = math.nan
    for score in ("softmax", "sigmoid"):
        check(high, 4, score=score)
        check(high, 4, score=score, bias=torch.zeros(E, device="cuda"))
    bias = torch.zeros(E, device="cuda")
    bias[9] = bias[4] = math.inf
    check(l.clamp(-12, 12), 4, score="sigmoid", bias=bias)
    bias[2] = math.nan
    check(l, 4, score="sigmoid", bias=bias)


def test_strided_rows_and_larger_counts():
    big, g = draw(5000, 300, 21)
    view = big[:, 17:17 + 96]
    bias = 0.1 * torch.randn(96, generator=g, device="cuda")
    a = R.route_select(view, 6, bias=bias, score="sigmoid", renorm=True)
    b = R.route_select(view.contiguous(), 6, bias=bias, score="sigmoid", renorm=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(view[:300], 6, bias=bias, score="sigmoid", renorm=True)
    empty = R.route_select(big[:0, :64], 6)
    assert empty[0].shape == (0, 6)


def test_stream_and_graph():
    """On a stream of its own and captured: the same bits, replayed with new inputs."""
    logits, g = draw(513, 64, 2)
    want = R.route_select(logits, 6, renorm=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = R.route_select(logits, 6, renorm=True)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    src = logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = R.route_select(src, 6, renorm=True)
    src.copy_(logits.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0].flip(0)) and torch.equal(out[1], want[1].flip(0))
