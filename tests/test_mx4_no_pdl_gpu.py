"""AFD_CFG_MX4 with AFD_CFG_NO_PDL: every kernel after the previous one has
finished, the same bits (narrow and wide products, token and grouped form)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from combine_peer_slot_gb300 import workloads as W


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def outputs(lens, grouped, flags):
    w = W.custom("fanin", seq_lens=lens, token_cap=2048)
    run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4 | flags, max_total_tokens=w.total_tokens)
    if grouped:
        run.prepare_grouped(seed=2)
        run.pack_grouped_all(0)
        assert run.forward_grouped(0) == 0
        ys, ss = run.unpack_grouped_all()
        out = [t.clone() for t in ys + ss]
    else:
        run.pack_all(0)
        assert run.forward(0) == 0
        out = [t.clone() for t in run.unpack_all()]
    assert run.poll() == 0
    run.close()
    return out


@pytest.mark.parametrize("lens", [[37, 91], [300, 450]])
@pytest.mark.parametrize("grouped", [False, True])
def test_same_bits_without_overlap(lens, grouped):
    a, b = outputs(lens, grouped, 0), outputs(lens, grouped, A.AFD_CFG_NO_PDL)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
