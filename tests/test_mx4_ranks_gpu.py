"""runtime.RankSet with its contexts in MXFP4: the experts split over ranks, each
with its block coded, against the 64-bit form of the step."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from combine_peer_slot_gb300 import workloads as W
from tests import test_mx4_forward_gpu as F


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


@pytest.mark.parametrize("ranks", [1, 3])
def test_ranks_take_the_flag(ranks):
    w = W.custom("fanin", seq_lens=[37, 91])
    rs = R.RankSet(w, ranks, flags=A.AFD_CFG_MX4)
    assert all(A.afd_get_workspace(c, A.AFD_WS_CODES)[1] > 0 for c in rs.ranks)
    rs.route()
    rs.dispatch_all()
    rs.serve_all()
    outs = rs.combine_all()
    assert rs.poll() == (0, 0)
    wt = rs.weights[0]
    for p, n in enumerate(w.seq_lens):
        xq = F.coded(rs.x[p])
        want = F.ffn64(xq, wt["W13s"], wt["Wds"])
        for e in range(w.num_experts):
            t, j = (rs.ids[p][:n] == e).nonzero(as_tuple=True)
            if t.numel():
                want[t] += rs.wts[p][t, j].double().unsqueeze(1) * F.ffn64(xq[t], wt["W13"][e], wt["Wd"][e])
        # the ranks' outputs travel in bf16: another 2^-8 of each term
        assert float((outs[p][:n].double() - want).norm() / want.norm()) <= F.TOL + 2.0 ** -8
    rs.close()
