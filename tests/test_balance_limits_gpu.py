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
