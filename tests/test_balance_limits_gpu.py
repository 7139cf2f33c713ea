"""The load's loss and the choice's gradient where their ranges end, against
64-bit forms."""
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


def test_sigmoids_below_64_bits():
    """Where exp(-l) leaves fp64, from -709.79 on, a sigmoid is 0, as in route_select:
    no share, no weight, no gradient; logits above that keep theirs beside it."""
    E, k = 48, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    l = torch.randn(24, E, generator=g, device="cuda")
    lowest = torch.finfo(torch.float32).min
    far = [-1e30, lowest, -709.8, -720.0, -760.0, -1e4]
    for i, v in enumerate(far):
        l[i] = v
        l[6 + i, ::3] = v                       # some
        l[12 + i] = v
        l[12 + i, 7] = -650.0                   # all but one, which is far down itself
        l[18 + i] = -709.7 + 0.05 * l[18 + i]   # around the border
        l[18 + i, 5:9] = v
    off = torch.arange(25, device="cuda").int()
    for same in (False, True):  # the choice, and one of the far entries alone
        ids, w = R.route_select(l, k, score="sigmoid", renorm=True)
        if same:
            ids = (torch.arange(k, device="cuda").int() + 5).repeat(24, 1)
            w = ref.weights(l.double(), ids, "sigmoid", True, 1.0)
        loss, counts = R.balance_loss(l, ids, score="sigmoid", seq_offsets=off)
        want, _ = ref.balance(l, ids, "sigmoid", off.tolist())
        assert ((loss.double() - want).abs() <= 100 * U * want).all()
        assert (loss[:6] == 0).all()
        dw = torch.randn(24, k, generator=g, device="cuda")
        d_loss = torch.randn(24, generator=g, device="cuda")
        for renorm in (False, True):
            for kw in (dict(d_weights=dw), dict(counts=counts, d_loss=d_loss), dict(d_weights=dw, counts=counts, d_loss=d_loss)):
                d = R.route_backward(l, ids, score="sigmoid", renorm=renorm, **kw, **({"seq_offsets": off} if "counts" in kw else {}))
                r, size = ref.route_grad(l, ids, "sigmoid", renorm=renorm, **kw, **({"offsets": off.tolist()} if "counts" in kw else {}))
                # (|l - top| up to 70 where it is not none)
                assert ((d.double() - r).abs() <= 300 * U * size + 1e-38).all()
        none = (w == 0).all(1)
        assert bool(none[:6].all())
        d = R.route_backward(l, ids, d_weights=dw, score="sigmoid", renorm=True)
        assert (d[none] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,T", [(256, 400000), (60, 700000)])
def test_one_long_sequence_among_many(score, E, T):
    """Nearly all rows in one of 400 sequences: however many rows a block adds up, its
    sums are off by at most 64 U of a row's shares (the exponential and its quotient), 64
    terms in fp32, and what warps and lanes add: 21."""
    S = 400
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    row = torch.randn(1, E, generator=g, device="cuda")
    l = row.repeat(T, 1)  # (equal rows: roundings of one sign, as an even gate's)
    ids = torch.full((T, 1), 3, dtype=torch.int32, device="cuda")
    off = torch.cat([torch.arange(200), torch.arange(T - 200, T + 1)]).int().cuda()
    assert off.numel() == S + 1
    loss, counts = R.balance_loss(l, ids, score=score, seq_offsets=off)
    _, p = ref.shares(row.double(), score)
    want = E * p[0, 3]  # of every sequence: E / n^2 n n p
    assert int(counts.sum()) == T and int(counts[199, 3]) == T - 399
    worst = float(((loss.double() - want) / want).abs().max())
    assert worst <= (64 + 64 + 21) * U, worst / U


@pytest.mark.parametrize("E", [33, 64, 100, 129, 256])
def test_many_rows_from_several_streams(E):
    """Losses of many rows, whose sums clusters of blocks finish, asked for again and
    again from four streams at a time: equal bits, and the 64-bit form's values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    l = torch.randn(5000, E, generator=g, device="cuda")
    ids, _ = R.route_select(l, 6)
    off = torch.tensor([0, 1, 1700, 1700, 4999, 5000], dtype=torch.int32, device="cuda")
    first, counts = R.balance_loss(l, ids, seq_offsets=off)
    want, wc = ref.balance(l, ids, "softmax", off.tolist())
    # (a share 64 U; at most 4999 / 64 rows in a chain)
    assert torch.equal(counts, wc) and ((first.double() - want).abs() <= 160 * U * want).all()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(50):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(R.balance_loss(l, ids, seq_offsets=off))
    torch.cuda.synchronize()
    assert all(torch.equal(a, first) and torch.equal(b, counts) for a, b in got)
