"""The adapters' first product over long rows of few tiles."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R

U = 2.0 ** -24


@pytest.mark.parametrize("dtype,steps", [(torch.bfloat16, 1), (torch.float32, 3)])
@pytest.mark.parametrize("rank", [1, 40])
def test_long_rows_of_many_adapters(dtype, steps, rank):
    """65536 columns of one sign, a tile a CTA: a warp's share is 256 chunks of 32
    columns, two MMAs each for a part of the rows.  The tensor cores' sums may cut 2 U
    a step; they move on every eight chunks, into sums that round, U each."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, K = 600, 65536
    g = torch.Generator(device="cuda")
    g.manual_seed(rank)
    ids = torch.arange(T, device="cuda").int()
    x = (1 + torch.rand(T, K, generator=g, device="cuda")).to(dtype)
    a = (1 + torch.rand(T, rank, K, generator=g, device="cuda", dtype=torch.bfloat16))
    b = torch.ones(T, rank, 8, dtype=torch.bfloat16, device="cuda")
    u = R.lora_apply(R.LoraBatch(ids, T), x, a, b, out_dtype=torch.float32, keep=True)[1]
    want = torch.stack([a[t].double() @ x[t].double() for t in range(T)])
    tol = (8 * 2 * steps * 2 + 256 / 8 + 8 + 8) * U
    worst = float(((u.double() - want) / want).abs().max())
    assert worst <= tol, worst / U
