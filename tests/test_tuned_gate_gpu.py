"""The tuning of a gate as a user runs it: logits of a shared gate with each
request's adapter beside it, the choice, its weights and the balance loss,
and back to the adapters and the rows, against a 64-bit form by autograd and
against its differences."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import tuning_reference as ref


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


@pytest.mark.parametrize("T,H,E,k,rank,L", [(37, 96, 16, 3, 5, 3), (1400, 128, 60, 6, 8, 5)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_tuned_gate(T, H, E, k, rank, L, score, renorm):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, gate = r(T, H).bfloat16(), r(E, H) / H ** 0.5
    a, b = (r(L, rank, H) / H ** 0.5).bfloat16(), (r(L, rank, E) / rank ** 0.5).bfloat16()
    scale = r(L)
    ids = torch.randint(-1, L, (T,), generator=g, device="cuda").int()
    off = torch.tensor([0, T // 4, T // 4, T], dtype=torch.int32, device="cuda")
    cw, cl = r(T, k), 3 * r(3)
    cl[1] = 0

    batch = R.LoraBatch(ids, L)
    logits, u = R.lora_apply(batch, x, a, b, x.float() @ gate.T, scale=scale, keep=True)
    chosen, w = R.route_select(logits, k, score=score, renorm=renorm, routed_scaling=1.5)
    loss, counts = R.balance_loss(logits, chosen, score=score, seq_offsets=off)
    d_logits = R.route_backward(logits, chosen, d_weights=cw, score=score, renorm=renorm, routed_scaling=1.5,
                                counts=counts, d_loss=cl, seq_offsets=off)
    dx, da, db = R.lora_backward(batch, x, d_logits, u, a, b, d_base=(d_logits @ gate).to(x.dtype), scale=scale)

    def value(x, a, b):
        v = x @ gate.double().T
        for l in range(L):
            rows = (ids == l).nonzero().flatten()
            v = v.index_add(0, rows, float(scale[l]) * (x[rows] @ a[l].T @ b[l]))
        _, p = ref.shares(v, score)
        total = (ref.weights(v, chosen, score, renorm, 1.5) * cw.double()).sum()
        for s, (lo, hi) in enumerate(ref.sequences(T, off.tolist())):
            if hi > lo:
                f = counts[s].double() * E / (k * (hi - lo) ** 2)
                total = total + cl[s].double() * (p[lo:hi].sum(0) * f).sum()
        return total

    at = [t.double().requires_grad_() for t in (x, a, b)]
    total = value(*at)
    # weights and losses: scores off by under 100 U, logits by the adapters' sums (some 1e-6)
    own = (w.double() * cw.double()).sum() + (loss.double() * cl.double()).sum()
    assert abs(float(own - total.detach())) <= 2e-5 * float((w.double() * cw.double()).abs().sum() + (loss.double() * cl.double()).abs().sum())
    want = torch.autograd.grad(total, at)
    for got, exact, tol in zip((dx, da, db), want, (2.0 ** -7, 2e-5, 2e-5)):
        # dx: d_base rounded to bf16 and dx itself, half a step each, of values up to their sum
        n = exact.abs().amax()
        assert float((got.double() - exact).abs().amax()) <= tol * float(n)
    h = 1e-4
    for i, got in enumerate((dx, da, db)):
        way = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        with torch.no_grad():
            up, down = [t.detach().clone() for t in at], [t.detach().clone() for t in at]
            up[i] += h * way
            down[i] -= h * way
            slope = float(value(*up) - value(*down)) / (2 * h)
        size = float((got.double() * way).square().sum().sqrt())
        # the differences' own error h^2 of third derivatives; dx's roundings, independent
        assert abs(float((got.double() * way).sum()) - slope) <= (2.0 ** -6 if i == 0 else 1e-3) * size
