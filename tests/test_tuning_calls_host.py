"""What the wrappers of the load, the choice's gradient and the adapters refuse
besides wrong types and sizes (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B
from combine_peer_slot_gb300 import runtime as R


@pytest.fixture(scope="module", autouse=True)
def lib():
    if B.needs_build():
        B.build()
    return A.lib()


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def code(fn, *a, **kw):
    with pytest.raises(A.AfdError) as e:
        fn(*a, **kw)
    return e.value.code


def test_a_loss_without_ids_has_no_topk():
    """The loss is divided by the choice's columns, so its gradient needs the ids'."""
    l, ids, counts = meta(4, 64), meta(4, 6, dtype=torch.int32), meta(1, 64, dtype=torch.int32)
    kw = dict(counts=counts, d_loss=meta(1))
    assert code(R.route_backward, l, None, **kw) == A.AFD_ERR_ARG
    assert code(R.route_backward, l, ids, **kw) == A.AFD_ERR_NOT_DEVICE
    assert code(R.route_backward, l, None) == A.AFD_ERR_NOT_DEVICE
