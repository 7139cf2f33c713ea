"""What the torch wrappers refuse before the library is called: tensors whose
memory is not what their sizes say, sizes that an int does not hold (no GPU
needed: the large tensors have no memory).  What is in range is refused later,
as no device memory."""
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


def meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device="meta")


WRAP = 2 ** 32


@pytest.mark.parametrize("bad", [dict(topk=WRAP + 6), dict(topk=6 - WRAP), dict(n_groups=WRAP + 1),
                                 dict(n_groups=8, topk_groups=WRAP + 4), dict(group_top=WRAP + 1), dict(topk=0)])
def test_select_sizes_do_not_wrap(bad):
    refused(A.AFD_ERR_ARG, R.route_select, meta(4, 64, dtype=torch.float32), **{"topk": 6, **bad})


def test_select_rows_and_experts_do_not_wrap():
    refused(A.AFD_ERR_ARG, R.route_select, meta(WRAP + 5, 64, dtype=torch.bfloat16), 6)
    refused(A.AFD_ERR_ARG, R.route_select, meta(2, WRAP + 64, dtype=torch.bfloat16), 6)
    refused(A.AFD_ERR_NOT_DEVICE, R.route_select, meta(4, 256, dtype=torch.bfloat16), 16, n_groups=32, topk_groups=2)


def test_coding_sizes_do_not_wrap():
    refused(A.AFD_ERR_ARG, R.mx4_quantize, meta(2, WRAP + 64, dtype=torch.bfloat16))
    refused(A.AFD_ERR_ARG, R.mx4_quantize, meta(2, 64, dtype=torch.bfloat16), topk=WRAP + 1)
    refused(A.AFD_ERR_NOT_DEVICE, R.mx4_quantize, meta(2, 65536, dtype=torch.bfloat16))
    refused(A.AFD_ERR_ARG, R.Mx4, meta(2, WRAP // 2 + 16), meta(2, WRAP // 32 + 1))
    assert R.Mx4(meta(2, 32768), meta(2, 2048)).cols == 65536


def test_weight_sizes_do_not_wrap():
    refused(A.AFD_ERR_ARG, R.Mx4Weight, meta(1, WRAP + 128, 64), meta(1, WRAP + 128, 4))
    refused(A.AFD_ERR_ARG, R.Mx4Weight, meta(1, 128, WRAP // 2 + 64), meta(1, 128, WRAP // 32 + 4))
    refused(A.AFD_ERR_ARG, R.Mx4Weight, meta(WRAP + 1, 128, 64), meta(WRAP + 1, 128, 4))
    refused(A.AFD_ERR_NOT_DEVICE, R.Mx4Weight, meta(1, 128, 64), meta(1, 128, 4))
