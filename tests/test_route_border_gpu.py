"""The routing choice with a bias where equal experts stand on both sides of
the border: the index decides between those, but a third expert whose exact
value is larger may share their fp32 value.  Ids are those of the 64-bit form;
a weight's bound is 64 units of 2^-24 of itself (the score 31 at most, the sum of
16, the division, the scaling)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import mx4_reference as ref


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def check(logits, topk, **kw):
    ids, w = R.route_select(logits, topk, **kw)
    rid, rw = ref.select(logits, topk, **kw)
    assert torch.equal(ids.cpu(), rid), (ids.cpu() != rid).any(1).nonzero().flatten()[:5]
    assert float(((w.double().cpu() - rw).abs() - 64 * 2.0 ** -24 * rw.abs()).max()) <= 1e-45
    return ids


def test_larger_score_behind_two_equal_ones():
    # three scores of 1.0f: only the exact ones differ
    ids = check(torch.tensor([[20.0, 20.0, 24.0]], device="cuda"), 1, bias=torch.zeros(3, device="cuda"), score="sigmoid")
    assert ids.tolist() == [[2]]
    # c = 1 + e-10 and less, in fp32 all 1
    ids = check(torch.tensor([[3.0, -20.0, -20.0, -18.0]], device="cuda"), 2, bias=torch.ones(4, device="cuda"))
    assert ids.tolist() == [[0, 3]]
    # several equal ones before the larger, in the same lane and in others
    for E in (8, 70, 200):
        for at in (E - 1, E // 2):
            row = torch.full((1, E), 18.0, device="cuda")
            row[0, at] = 19.0
            ids = check(row, 1, bias=torch.full((E,), 0.5, device="cuda"), score="sigmoid")
            assert ids.tolist() == [[at]]
            check(row, 3, bias=torch.full((E,), 0.5, device="cuda"), score="sigmoid")
    # equal logits, another bias of the same fp32 sum
    bias = torch.tensor([2.0 ** -25, 2.0 ** -25, 2.0 ** -25 * (1 + 2.0 ** -20), 0.0], device="cuda")
    check(torch.full((1, 4), 20.0, device="cuda"), 1, bias=bias, score="sigmoid")


@pytest.mark.parametrize("E,k", [(64, 6), (128, 3), (256, 8), (61, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [1.5, 8.0])  # 8: scores that saturate
def test_repeated_logits(E, k, score, spread):
    """bf16 logits on a coarse grid, few biases: many equal experts in every row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(E + k)
    logits = ((spread * torch.randn(150, E, generator=g, device="cuda")) * 2).round() / 2
    logits += (torch.rand(150, E, generator=g, device="cuda") < 0.1) * 0.25
    for bias in (torch.zeros(E, device="cuda"), torch.ones(E, device="cuda"),
                 torch.randint(0, 2, (E,), generator=g, device="cuda").float()):
        for dtype in (torch.bfloat16, torch.float32):
            check(logits.to(dtype), k, bias=bias, score=score)
            check(logits.to(dtype), k, bias=bias, score=score, renorm=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_repeated_logits_in_groups(score):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = (8 * torch.randn(150, 64, generator=g, device="cuda")).round()
    for group_top in (1, 2):
        check(logits, 4, bias=torch.zeros(64, device="cuda"), score=score, n_groups=8, topk_groups=3, group_top=group_top)


def test_infinite_biases():
    """Several biases of +inf and -inf: the index decides between equal infinities."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    logits = torch.randn(40, 33, generator=g, device="cuda").round()
    bias = torch.zeros(33, device="cuda")
    bias[[4, 9, 20, 31]] = float("inf")
    bias[[0, 11]] = -float("inf")
    for k in (1, 2, 4, 5):
        check(logits, k, bias=bias, score="sigmoid")
