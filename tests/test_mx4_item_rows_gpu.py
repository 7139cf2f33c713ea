"""A step of the work-item loop codes its own rows, not the context's capacity
(AFD_CFG_MX4): codes behind the step's last row stay as they were, and the
outputs are those of the host-described step."""
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


@pytest.mark.parametrize("shared", [64, 0])
@pytest.mark.parametrize("counts", [[3, 4], [0, 1], [37, 91], [0, 0]])
def test_codes_behind_the_step_stay(counts, shared):
    w = W.custom("fanin", seq_lens=[37, 91], layers=1, token_cap=2048, shared_inter=shared)
    run = R.Runner(w, layers=1, ring_depth=2, flags=A.AFD_CFG_MX4, max_total_tokens=4096)
    codes = run.workspace(A.AFD_WS_CODES).view(-1, w.hidden // 2)
    assert codes.shape[0] == 4096 * (w.topk + 1)

    def pack():
        seqs = []
        for p, n in enumerate(counts):
            run.seq += 1
            rc = A.afd_pack_slot(run.ctx, p, 0, 0, run.x[p].data_ptr() if n else 0, n, shared > 0, run.seq)
            assert rc == 0
            seqs.append(run.seq)
        return seqs

    def unpack(seqs):
        for p, n in enumerate(counts):
            assert A.afd_unpack_split(run.ctx, p, 0, run.out[p].data_ptr() if n else 0, n, seqs[p]) == 0
        assert run.poll() == 0
        return [run.out[p][:n].clone() for p, n in enumerate(counts)]

    codes.fill_(0xAB)
    torch.cuda.synchronize()
    seqs = pack()
    assert A.afd_ffn_serve(run.ctx, [0, 1], 1) == 0
    got = unpack(seqs)
    rows = sum(counts) * (w.topk + (1 if shared else 0))
    assert bool((codes[rows:] == 0xAB).all())
    coded = codes[:rows].clone()
    seqs = pack()
    assert A.afd_ffn_forward(run.ctx, 0, 0, counts, [0, 1]) == 0
    want = unpack(seqs)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(codes[:rows], coded)
    run.close()


def test_no_codes_without_the_flag():
    run = R.Runner(W.custom("fanin", seq_lens=[3, 4]), layers=1)
    assert A.afd_get_workspace(run.ctx, A.AFD_WS_CODES)[1] == 0
    run.close()


def test_no_uncoded_swiglu_rows_with_the_flag():
    """The SwiGLU rows exist as codes only: no workspace for bf16 ones."""
    w = W.custom("fanin", seq_lens=[3, 4])
    for flags, bytes_ in ((A.AFD_CFG_MX4, 0), (0, 2)):
        run = R.Runner(w, layers=1, flags=flags, max_total_tokens=64)
        assert A.afd_get_workspace(run.ctx, A.AFD_WS_H)[1] == 64 * w.topk * w.inter * bytes_
        assert A.afd_get_workspace(run.ctx, A.AFD_WS_HS)[1] == 64 * w.shared_inter * bytes_
        run.close()
