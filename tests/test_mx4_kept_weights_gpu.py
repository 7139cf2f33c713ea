"""Weights whose bf16 values are MXFP4 values already are kept exactly: the coder
picks each block's scale by its largest value, so a block whose largest code is
0.5 to 3 gets a smaller scale and larger codes, of the same values.  Values
made from random codes and scales, coded again; and a step on such weights
against a 64-bit form that uses the values as they are."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from combine_peer_slot_gb300 import workloads as W
from tests import mx4_reference as ref
from tests import test_mx4_forward_gpu as F

TOPS = [0, 1, 2, 3, 4, 5, 6, 7]  # the largest code a block may hold: 0, 0.5, 1, 1.5, 2, 3, 4, 6


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def foreign(shape, lo, hi, seed):
    """bf16 values of random codes, each block's limited to a random largest one,
    and random scale bytes lo .. hi."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    *rows, cols = shape
    top = torch.randint(0, len(TOPS), (*rows, cols // 32, 1), generator=g, device="cuda")
    mag = (torch.randint(0, 1 << 20, (*rows, cols // 32, 32), generator=g, device="cuda") % (top + 1)).flatten(-2)
    code = (mag + 8 * torch.randint(0, 2, (*rows, cols), generator=g, device="cuda")).to(torch.uint8)
    scale = torch.randint(lo, hi + 1, (*rows, cols // 32), generator=g, device="cuda").to(torch.uint8)
    v = ref.decode(code[..., 0::2] | (code[..., 1::2] << 4), scale)
    b = v.bfloat16()
    assert torch.equal(b.double(), v)  # three significant bits
    return b


@pytest.mark.parametrize("lo,hi", [(0, 8), (100, 140), (240, 252)])  # the smallest scales, usual ones, the largest
def test_values_code_to_themselves(lo, hi):
    w = foreign((500, 256), lo, hi, lo)
    for rule in ("floor", "ceil"):
        for x in (w, w.float()):
            q = R.mx4_quantize(x, rule=rule)
            for dt in (torch.bfloat16, torch.float32):
                assert torch.equal(R.mx4_dequantize(q, dt).double(), w.double())


def test_step_on_kept_weights():
    w = W.custom("fanin", seq_lens=[37, 91])
    run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4)
    E, H, I, S = w.num_experts, w.hidden, w.inter, w.shared_inter
    wt = {"W13": foreign((E, 2 * I, H), 119, 122, 1), "Wd": foreign((E, H, I), 119, 122, 2),
          "W13s": foreign((2 * S, H), 119, 122, 3), "Wds": foreign((H, S), 119, 122, 4)}
    A.afd_set_layer(run.ctx, 0, run.Wg.data_ptr(), run.bias.data_ptr() if run.bias is not None else 0,
                    *[wt[k].data_ptr() for k in ("W13", "Wd", "W13s", "Wds")])
    run.pack_all(0)
    assert run.forward(0) == 0
    outs = run.unpack_all()
    assert run.poll() == 0
    ids, gate = F.routing(run, w.total_tokens)
    xq = F.coded(torch.cat(run.x))

    def ffn(x, a, b):
        h = ref.swiglu(x @ a.double().T).bfloat16()
        return F.coded(h) @ b.double().T

    want = ffn(xq, wt["W13s"], wt["Wds"])
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            want[t] += gate[t, j].double().unsqueeze(1) * ffn(xq[t], wt["W13"][e], wt["Wd"][e])
    F.close(torch.cat(outs), want)
    run.close()
