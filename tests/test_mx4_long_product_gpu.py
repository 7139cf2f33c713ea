"""A product that takes longer than the bound on its waits (2 s each) ends like
any other: the bound is a wait's, not the kernel's.  The length comes from
groups that overlap (every second one covers all rows: such a call's outputs
are unspecified, here every writer of a row writes the same zeros) over 250 M rows
of one scale block, 10 GB in all."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("40 GB wanted")
    A.lib()


def test_longer_than_the_bound_of_a_wait():
    n, E, M, K = 250_000_000, 256, 8, 32
    w = R.Mx4Weight(torch.zeros(E, M, K // 2, dtype=torch.uint8, device="cuda"),
                    torch.full((E, M, 1), 127, dtype=torch.uint8, device="cuda"))
    x = R.Mx4(torch.zeros(n, K // 2, dtype=torch.uint8, device="cuda"),
              torch.full((n, 1), 127, dtype=torch.uint8, device="cuda"))
    off = torch.tensor([0, n] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    out = torch.full((n, M), 5.0, dtype=torch.bfloat16, device="cuda")
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    R.mx4_gemm(x, off, w, out=out)
    t1.record()
    torch.cuda.synchronize()
    assert A.afd_mx4_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK
    assert not bool(out.any())
    assert t0.elapsed_time(t1) > 2500.0  # the test's own premise
    del x, w, out
    torch.cuda.empty_cache()
