"""A step that has failed does no expert work (AFD_CFG_MX4): its products leave
the workspace as it was, whatever rows and weights an earlier step left there,
and the context works again afterwards.  The failures are made on the host: a
flag that nothing sets and a short bound on the wait."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from combine_peer_slot_gb300 import workloads as W

WAIT_NS = 20_000_000


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def outputs(run):
    return [run.workspace(A.AFD_WS_Y), run.workspace(A.AFD_WS_S)]


def fill(run):
    torch.cuda.synchronize()
    for t in outputs(run):
        t.fill_(0xAB)
    torch.cuda.synchronize()


def untouched(run):
    return all(bool((t == 0xAB).all()) for t in outputs(run))


@pytest.mark.parametrize("lens", [[20, 30], [300, 450]])  # the narrow and the wide products
def test_timed_out_step_leaves_the_outputs(lens):
    run = R.Runner(W.custom("fanin", seq_lens=lens), layers=1, flags=A.AFD_CFG_MX4, wait_timeout_ns=WAIT_NS)
    run.pack_all(0)
    assert run.forward(0) == 0
    want = [o.clone() for o in run.unpack_all()]
    assert run.poll() == 0
    fill(run)
    assert run.forward(0) == 0            # the flags never advance
    assert run.forward(0) == 0            # queued behind the failed one
    assert run.poll() == A.AFD_ERR_TIMEOUT
    assert untouched(run)
    run.pack_all(0)
    assert run.forward(0) == 0
    got = run.unpack_all()
    assert run.poll() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    run.close()


@pytest.mark.parametrize("lens", [[20, 30], [300, 450]])
def test_item_that_never_comes(lens, monkeypatch):
    """The loop's first item does not come, and layer 0, which an item not yet
    written names, has no weights; an earlier host-described step has left rows."""
    real = A.afd_set_layer
    monkeypatch.setattr(A, "afd_set_layer", lambda ctx, layer, *a: None if layer == 0 else real(ctx, layer, *a))
    w = W.custom("fanin", seq_lens=lens, layers=2)
    run = R.Runner(w, layers=2, flags=A.AFD_CFG_MX4, wait_timeout_ns=WAIT_NS, ring_depth=2,
                   max_total_tokens=w.total_tokens)
    run.pack_all(1)
    assert run.forward(1) == 0
    want = [o.clone() for o in run.unpack_all()]
    assert run.poll() == 0
    fill(run)
    assert A.afd_ffn_serve(run.ctx, [0, 1], 2) == 0
    assert run.poll() == A.AFD_ERR_TIMEOUT
    assert untouched(run)
    run.pack_all(1)
    assert A.afd_ffn_serve(run.ctx, [0, 1], 1) == 0
    got = run.unpack_all()
    assert run.poll() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    run.close()
