"""afd_balance_loss and afd_route_backward against plain 64-bit forms: counts
equal, losses and gradients within what fp32 arithmetic may be off.

A share p is off by at most 64 U of itself (the exponential's 2 and its
argument's rounding, |l - top| <= 24 here: 24; the sum over 256 lanes' terms
8 + 5; the division 2), a sum of shares by a step more for each term of its
longest chain; a gradient is a difference of two such products, bounded term
by term in the reference: 160 U of that, and half a step of its type."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import tuning_reference as ref

U = ref.U


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def draw(T, E, k, seed, dtype=torch.float32, gone=0.0):
    g = gen(seed)
    l = 1.5 * torch.randn(T, E, generator=g, device="cuda")
    if gone:
        l.masked_fill_(torch.rand(T, E, generator=g, device="cuda") < gone, -math.inf)
    l = l.to(dtype)
    ids = R.route_select(l, k)[0]
    return l, ids, g


def check_balance(l, ids, score, off=None):
    loss, counts = R.balance_loss(l, ids, score=score, seq_offsets=off)
    want, wc = ref.balance(l, ids, score, off.tolist() if off is not None else None)
    assert torch.equal(counts, wc)
    S, E = wc.shape
    chunks = max(1, A.afd_balance_workspace(l.shape[0], E, S) // (8 * S * E))
    tol = (64 + l.shape[0] / (8 * chunks) + 16) * U
    assert torch.equal(torch.isnan(loss), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert ((loss.double() - want).abs()[fine] <= tol * want.abs()[fine]).all()
    return loss, counts


def check_grad(l, ids, score, out=None, **kw):
    kr = {("scaling" if k == "routed_scaling" else "offsets" if k == "seq_offsets" else k): v for k, v in kw.items()}
    if kr.get("offsets") is not None:
        kr["offsets"] = kr["offsets"].tolist()
    want, size = ref.route_grad(l, ids, score, **kr)
    d = R.route_backward(l, ids, score=score, out=out, **kw)
    assert d.dtype == l.dtype
    assert torch.equal(torch.isnan(d), torch.isnan(want))
    fine = ~torch.isnan(want)
    tol = 160 * U * size + ref.HALF[l.dtype] * (want.abs() + 160 * U * size) + 1e-38
    assert ((d.double() - want).abs()[fine] <= tol[fine]).all()
    return d


SIZES = [(1, 1, 1, 1), (1, 64, 6, 1), (2, 2, 2, 3), (37, 60, 4, 5), (9, 33, 16, 2), (329, 64, 6, 16), (512, 128, 8, 3),
         (513, 129, 7, 2), (700, 100, 3, 40), (1999, 255, 5, 1), (4000, 256, 16, 7), (2500, 8, 2, 64)]


@pytest.mark.parametrize("T,E,k,S", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(T, E, k, S, score, dtype):
    l, ids, g = draw(T, E, k, T + E, dtype, gone=0.1 if T % 2 else 0.0)
    cut = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values.int()
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)])
    _, counts = check_balance(l, ids, score, off)
    d_loss = torch.randn(S, generator=g, device="cuda")
    dw = torch.randn(T, k, generator=g, device="cuda")
    check_grad(l, ids, score, counts=counts, d_loss=d_loss, seq_offsets=off)
    for renorm in (False, True):
        check_grad(l, ids, score, d_weights=dw, renorm=renorm, routed_scaling=2.5)
        check_grad(l, ids, score, d_weights=dw, renorm=renorm, counts=counts, d_loss=d_loss, seq_offsets=off)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [300, 3000])
def test_sequences(score, T):
    """Empty sequences, rows before the first and behind the last, no offsets."""
    l, ids, g = draw(T, 48, 6, 5)
    off = torch.tensor([7, 7, 40, 40, T - 30], dtype=torch.int32, device="cuda")
    loss, counts = check_balance(l, ids, score, off)
    assert float(loss[0]) == 0.0 == float(loss[2]) and int(counts[0].sum()) == 0
    d_loss = torch.randn(4, generator=g, device="cuda")
    d = check_grad(l, ids, score, counts=counts, d_loss=d_loss, seq_offsets=off)
    assert (d[:7] == 0).all() and (d[T - 30:] == 0).all()
    check_balance(l, ids, score)
    past = torch.tensor([-5, 10, T + 100], dtype=torch.int32, device="cuda")  # clamped to the rows
    check_balance(l, ids, score, past)
    even, c = R.balance_loss(torch.zeros(T, 8, device="cuda"), torch.arange(T, device="cuda").view(-1, 1).int() % 8,
                             score=score)
    if T % 8 == 0:
        assert abs(float(even[0]) - 1) < 1e-5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [60, 900])
def test_masked_and_repeated(score, T):
    """Rows with few experts left, one, none; ids of no choice, out of range, twice in a row."""
    l, _, g = draw(T, 40, 6, 9)
    gone = torch.rand(T, 40, generator=g, device="cuda") < torch.linspace(0, 1.05, T, device="cuda").unsqueeze(1)
    l[gone] = -math.inf
    l[0] = -math.inf
    l[1, :39] = -math.inf
    ids = R.route_select(l, 6)[0]
    ids[5] = torch.tensor([3, 3, 3, -1, 7, 3], device="cuda").int()
    ids[6] = torch.tensor([-7, 40, 2 ** 30, -1, 0, 39], device="cuda").int()
    _, counts = check_balance(l, ids, score)
    d_loss = torch.full((1,), 0.7, device="cuda")
    dw = torch.randn(T, 6, generator=g, device="cuda")
    for renorm in (False, True):
        check_grad(l, ids, score, d_weights=dw, renorm=renorm, counts=counts, d_loss=d_loss)
    dw[ids < 0] = math.nan  # what stands beside no choice is not read into a sum
    d = R.route_backward(l, ids, d_weights=dw, score=score, renorm=True)
    assert not torch.isnan(d).any()
    assert (R.route_backward(l, ids, d_weights=dw, score=score, counts=counts, d_loss=d_loss)[0] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extremes(score):
    """NaN and infinite logits, far apart and far below, without a part's inputs."""
    T, E, k = 24, 64, 4
    l, ids, g = draw(T, E, k, 3)
    l[1, 5] = math.nan
    l[2, 7] = math.inf
    l[3] = -200.0 + l[3]
    l[4] = -1e30
    l[5, 0] = 3e38
    l[6] = 80.0 + l[6]
    l[7, :32] = -math.inf
    ids = ids.clone()
    ids[8] = torch.tensor([60, 61, 62, 63], device="cuda").int()
    l[8, 60:] = l[8, :60].min() - 150 + torch.arange(4, device="cuda")  # chosen far below the rest
    off = torch.arange(T + 1, device="cuda").int()
    loss, counts = R.balance_loss(l, ids, score=score, seq_offsets=off)
    want, _ = ref.balance(l, ids, score, off.tolist())
    nan = torch.isnan(loss)
    assert bool(nan[1]) and bool(nan[2]) == (score == "softmax") and int(nan.sum()) == 1 + (score == "softmax")
    ok = ~nan
    ok[4] = False  # (sigmoids of -1e30: 0 in any precision, shares of the softmax here)
    # (row 5's choices other than the one with all the mass have losses of 1e-67, which fp32 does not hold: the
    # last term is its smallest normal number)
    assert ((loss.double() - want)[ok].abs() <= 100 * U * want[ok] + 2.0 ** -126).all()
    dw = torch.randn(T, k, generator=g, device="cuda")
    keep = [t for t in range(T) if t != 4]
    for renorm in (False, True):
        d = R.route_backward(l, ids, d_weights=dw, score=score, renorm=renorm)
        w, size = ref.route_grad(l, ids, score, d_weights=dw, renorm=renorm)
        assert torch.equal(torch.isnan(d)[keep], torch.isnan(w)[keep])
        tol = 400 * U * size + 1e-38  # (|l - top| up to 174 here)
        e = (d.double() - w).abs() - tol
        assert (e[keep][~torch.isnan(w)[keep]] <= 0).all()
    zero = R.route_backward(l, None, score=score)
    assert (zero[0] == 0).all() and torch.isnan(zero[1]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides(dtype):
    """Row pitches that are and are not whole runs, out of another pitch, out = logits."""
    for pitch, first in ((64, 0), (72, 8), (67, 1), (61, 0)):
        wide, ids, g = draw(333, pitch, 5, pitch, dtype)
        l = wide[:, first:first + 60]
        ids = R.route_select(l, 5)[0]
        _, counts = check_balance(l, ids, "softmax")
        dw = torch.randn(333, 5, generator=g, device="cuda")
        store = torch.full((333, 75), 7.0, dtype=dtype, device="cuda")
        kw = dict(d_weights=dw, renorm=True, counts=counts, d_loss=torch.ones(1, device="cuda"))
        d = check_grad(l, ids, "softmax", out=store[:, 3:63], **kw)
        assert (store[:, :3] == 7).all() and (store[:, 63:] == 7).all()
        own = wide.clone()
        view = own[:, first:first + 60]
        assert torch.equal(R.route_backward(view, ids, out=view, **kw), d)


def test_offsets_over_32_bits():
    T, pitch = 700, (5 * 2 ** 29) // 700 // 8 * 8
    l = torch.empty(T * pitch, dtype=torch.bfloat16, device="cuda").view(T, pitch)[:, :64]
    l.copy_(draw(T, 64, 6, 1, torch.bfloat16)[0])
    ids = R.route_select(l, 6)[0]
    _, counts = check_balance(l, ids, "softmax")
    check_grad(l, ids, "softmax", counts=counts, d_loss=torch.ones(1, device="cuda"))


def test_many_sequences():
    """As many sequences as rows, more, and more than there are shares of the sums."""
    for T, S in ((600, 600), (2000, 3000), (900, 400)):
        l, ids, g = draw(T, 32, 4, S)
        cut = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values.int()
        off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)])
        _, counts = check_balance(l, ids, "sigmoid", off)
        check_grad(l, ids, "sigmoid", counts=counts, d_loss=torch.randn(S, generator=g, device="cuda"), seq_offsets=off)


def test_no_rows():
    l = torch.zeros(0, 8, device="cuda")
    ids = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, counts = R.balance_loss(l, ids, seq_offsets=off)
    assert (loss == 0).all() and (counts == 0).all()
    assert R.route_backward(l, ids, d_weights=torch.zeros(0, 2, device="cuda")).shape == (0, 8)


@pytest.mark.parametrize("T", [200, 5000])
def test_repeats_and_graphs(T):
    """Equal bits from call to call, on another stream, and from a replayed graph on new logits."""
    l, ids, g = draw(T, 96, 6, 2)
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    dl = torch.ones(2, device="cuda")

    def both():
        loss, counts = R.balance_loss(l, ids, seq_offsets=off)
        return loss, counts, R.route_backward(l, ids, counts=counts, d_loss=dl, seq_offsets=off)

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    other, oids, _ = draw(T, 96, 6, 77)
    l.copy_(other)
    ids.copy_(oids)
    graph.replay()
    again = both()
    assert all(torch.equal(a, b) for a, b in zip(held, again)) and not torch.equal(again[0], first[0])
