"""The work-item loop when its first item never comes and layer 0 has no
weights: an item that was not written names layer 0, so nothing of the step may
follow that name to memory.  The failure is a flag that nothing sets and a short
bound on the wait."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from combine_peer_slot_gb300 import workloads as W

ENGINES = [A.AFD_GEMM_TENSOR, A.AFD_GEMM_TENSOR_1CTA, A.AFD_GEMM_SIMT]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


@pytest.mark.parametrize("gemm", ENGINES)
@pytest.mark.parametrize("earlier", [False, True])  # a host-described step before
def test_first_item_never_comes_and_layer_0_is_not_set(gemm, earlier, monkeypatch):
    real = A.afd_set_layer
    monkeypatch.setattr(A, "afd_set_layer", lambda ctx, layer, *a: None if layer == 0 else real(ctx, layer, *a))
    w = W.custom("fanin", seq_lens=[20, 30], layers=2)
    run = R.Runner(w, layers=2, gemm=gemm, wait_timeout_ns=20_000_000, ring_depth=2, max_total_tokens=w.total_tokens)
    if earlier:
        run.pack_all(1)
        assert run.forward(1) == 0
        run.unpack_all()
        assert run.poll() == 0
    assert A.afd_ffn_serve(run.ctx, [0, 1], 2) == 0
    assert run.poll() == A.AFD_ERR_TIMEOUT
    run.pack_all(1)
    assert A.afd_ffn_serve(run.ctx, [0, 1], 1) == 0
    got = [o.clone() for o in run.unpack_all()]
    assert run.poll() == 0
    run.pack_all(1)
    assert run.forward(1) == 0
    want = run.unpack_all()
    assert run.poll() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    run.close()
