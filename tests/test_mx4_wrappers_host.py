"""What the torch wrappers refuse before the library is called: tensors whose
memory is not what their sizes say (no GPU needed)."""
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


def refused(code, fn, *a, **kw):
    with pytest.raises(A.AfdError) as e:
        fn(*a, **kw)
    assert e.value.code == code


@pytest.mark.parametrize("make", [lambda t: t[:1].expand(1 << 20), lambda t: t[::2], lambda t: t.view(64, 64).t()])
def test_workspace_is_one_run_of_memory(make):
    h = R._get()
    whole = torch.zeros(4096, dtype=torch.uint8)
    refused(A.AFD_ERR_ARG, R._scratch, h, make(whole), 1024, whole.device)
    assert R._scratch(h, whole, 1024, whole.device)[:2] == (whole.data_ptr(), 4096)
    f = torch.zeros(64, 16)
    assert R._scratch(h, f, 1024, f.device)[:2] == (f.data_ptr(), 4096)
