"""The sizes that the MXFP4 queries answer are those that the calls take (no GPU needed)."""
import pytest

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B

P = 0x10000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if B.needs_build():
        B.build()
    return A.lib()


@pytest.mark.parametrize("hidden,inter,ok", [(128, 32768, True), (128, 32800, False), (128, 40000, False),
                                             (128, 65536, False), (65536, 32768, True), (65568, 64, False),
                                             (96, 64, True), (100, 64, False), (32, 32, True)])
def test_ffn_workspace_and_call_agree(hidden, inter, ok):
    n = A.afd_mx4_ffn_workspace(4, 2, hidden, inter)
    assert (n > 0) == ok and (ok or n == -1)
    both = (A.afd_mx4_weight_bytes(2, 2 * inter, hidden, True) > 0 and A.afd_mx4_weight_bytes(2, hidden, inter, False) > 0)
    assert both == ok
    call = dict(codes=P, scales=P, n_rows=4, offsets=P, num_experts=2, w13=P, wd=P, hidden=hidden, inter=inter,
                out_dtype=A.AFD_DTYPE_BF16, out=P, ldo=hidden + (-hidden) % 8, workspace=P)
    # too small a workspace is the answer for sizes that are taken
    want = A.AFD_ERR_CAPACITY if ok else A.AFD_ERR_ARG
    assert A.afd_mx4_ffn(**call, workspace_bytes=max(0, n - 1)) == want
