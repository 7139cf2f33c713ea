"""What a step of AFD_CFG_MX4 leaves in its workspace, bit for bit the calls it
stands for on the same rows: the gathered rows coded (mx4_quantize with the
step's permutation), the expert FFN of the routed rows in fp32 rounded to 24 bits
(AFD_WS_Y), that of the shared rows in fp32 (AFD_WS_S).  Those calls are held
to the 64-bit forms elsewhere."""
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


def coded(w, swiglu):
    w = w if w.dim() == 3 else w.unsqueeze(0)
    q = R.mx4_quantize(w.reshape(-1, w.shape[-1]))
    return R.Mx4Weight(q.codes.view(*w.shape[:2], -1), q.scales.view(*w.shape[:2], -1), swiglu=swiglu)


def ints(run, which, n):
    return run.workspace(which, 4 * n).view(torch.int32).clone()


@pytest.mark.parametrize("shape", [dict(seq_lens=[37, 91]), dict(seq_lens=[1, 0]), dict(seq_lens=[900, 1200]),
                                   dict(seq_lens=[77, 202], hidden=288, inter=96, shared_inter=160),
                                   dict(seq_lens=[700, 801], hidden=544, inter=352, shared_inter=96)])
def test_step_is_its_calls(shape):
    w = W.custom("fanin", **shape)
    run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4, max_total_tokens=w.total_tokens)
    run.pack_all(0)
    assert run.forward(0) == 0
    assert run.poll() == 0
    T, k, H, E = w.total_tokens, w.topk, w.hidden, w.num_experts
    N = T * k
    perm, off = ints(run, A.AFD_WS_PERM, N), ints(run, A.AFD_WS_OFFSETS, E + 1)
    x = torch.cat([t[:n] for t, n in zip(run.x, w.seq_lens)])
    wt = run.weights[0]
    q = R.mx4_quantize(x, src_rows=perm, topk=k)
    codes = run.workspace(A.AFD_WS_CODES, (N + T) * H // 2).view(N + T, H // 2)
    assert torch.equal(codes[:N], q.codes)
    y = R.mx4_ffn(q, off, coded(wt["W13"], True), coded(wt["Wd"], False), out_dtype=torch.float32)
    # 24 bits: the low 8 rounded off, half away from zero
    bits = (y.view(torch.int32) + 0x80) >> 8
    raw = run.workspace(A.AFD_WS_Y)
    hi = raw[:2 * N * H].view(torch.int16).view(N, H)
    low0 = raw.numel() // 2  # the low plane follows the high plane's capacity (2 + 1 of 4 bytes a value)
    lo = raw[low0:low0 + N * H].view(N, H)
    assert torch.equal(hi.int() & 0xFFFF, (bits >> 8) & 0xFFFF)
    assert torch.equal(lo.int(), bits & 0xFF)
    shared = R.mx4_quantize(x)
    assert torch.equal(codes[N:], shared.codes)
    s = R.mx4_ffn(shared, torch.tensor([0, T], dtype=torch.int32, device="cuda"), coded(wt["W13s"], True),
                  coded(wt["Wds"], False), out_dtype=torch.float32)
    assert torch.equal(run.workspace(A.AFD_WS_S, 4 * T * H).view(torch.float32).view(T, H), s)
    run.close()
