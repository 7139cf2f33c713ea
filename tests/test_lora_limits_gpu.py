"""The adapters' calls where their arithmetic and their pipelines reach furthest,
against 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import test_lora_gpu as form

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def digits(T, cols, g):
    """Rows whose first three values h, m, l add up to 24 bits, 8 of them each."""
    x = torch.zeros(T, cols, device="cuda")
    for i in range(3):
        x[:, i] = torch.randint(128, 256, (T,), generator=g, device="cuda").float() / 128 * 2.0 ** (-8 * i)
    return x


def pairs(rank, src, out):
    """Weights for which even ranks hold h + m + l, odd ones h + m, and each output is one even rank less the next odd one."""
    w1, w2 = torch.zeros(2, rank, src, device="cuda"), torch.zeros(2, rank, out, device="cuda")
    w1[:, :, :2] = 1
    w1[:, ::2, 2] = 1
    p = 2 * (torch.arange(out, device="cuda") % (rank // 2))
    w2[:, p, torch.arange(out, device="cuda")] = 1
    w2[:, p + 1, torch.arange(out, device="cuda")] = -1
    return w1.to(BF), w2.to(BF)


@pytest.mark.parametrize("T,rank", [(40, 8), (40, 60), (1600, 16), (1600, 32), (1600, 48), (1600, 64), (1600, 100)])
@pytest.mark.parametrize("pitch", [64, 63])
def test_u_keeps_its_bits(T, rank, pitch):
    """Beside bf16 outputs u enters the second product with all of fp32's bits: the
    difference of two of its values that differ in the last eight comes out.  Off by
    at most: the first product's one step, 2 U of terms up to 2.02, for both; the
    second's three, 2 U of their 4.04 each: under 33 U.  The output's rounding, half
    a step of under 2^-15: 2^-23."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + rank)
    ids = torch.randint(0, 2, (T,), generator=g, device="cuda").int()
    x = torch.zeros(T, pitch, dtype=BF, device="cuda")[:, :56]
    x.copy_(digits(T, 56, g))
    low = x[:, 2:3].double()
    tol = 33 * U + 2.0 ** -23
    batch = R.LoraBatch(ids, 2)
    w1, w2 = pairs(rank, 56, 48)
    y, u = R.lora_apply(batch, x, w1, w2, keep=True)
    assert y.dtype == BF and ((y.double() - low).abs() <= tol).all()
    dx = R.lora_backward(batch, torch.zeros(T, 48, dtype=BF, device="cuda"), x, u, w2, w1)[0]
    assert dx.dtype == BF and ((dx.double() - low).abs() <= tol).all()


# Over 152 tiles, so that a persistent CTA goes from item to item (over 304: twice), over
# 1024 columns of both products, so that its ring wraps within each and every barrier
# is waited for; pieces times slabs of the weight gradients likewise, in each of its forms.
MANY = [(24000, 1096, 1160, 48, 200, "mixed"), (24000, 1160, 1096, 64, 400, "mixed"), (45000, 1096, 600, 64, 4, "runs"),
        (9000, 520, 2100, 100, 40, "mixed"), (9000, 2100, 520, 128, 12, "mixed"), (20000, 1032, 1096, 16, 300, "mixed"),
        (20000, 1096, 1032, 32, 90, "mixed")]


@pytest.mark.parametrize("T,K,M,rank,L,how", MANY)
def test_many_items_a_block(T, K, M, rank, L, how):
    d = form.make(T, K, M, rank, L, BF, BF, how, T + rank)
    batch, _, u = form.check_apply(d)
    form.check_backward(d, batch, u)
    assert A.afd_lora_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK


@pytest.mark.parametrize("T,rank,L", [(12000, 48, 160), (30000, 64, 9), (5000, 100, 60)])
def test_many_items_repeat(T, rank, L):
    """Equal bits from call to call, from two streams at a time with one plan, and from a
    replayed graph."""
    d = form.make(T, 1032, 712, rank, L, BF, BF, "mixed", rank)
    batch = R.LoraBatch(d["ids"], L)

    def both():
        y, u = R.lora_apply(batch, d["x"], d["a"], d["b"], d["base"], scale=d["scale"], keep=True)
        return (y, u) + R.lora_backward(batch, d["x"], d["dy"], u, d["a"], d["b"], d_base=d["d_base"], scale=d["scale"])

    first = both()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(both())
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in got for p, q in zip(o, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, first))
    assert A.afd_lora_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK


def test_tensors_that_ask_for_gradients():
    """Taken as values: equal bits, outputs without a graph, whose gradients are calls of their own."""
    d = form.make(40, 64, 96, 8, 3, BF, BF, "mixed", 2)
    batch = R.LoraBatch(d["ids"], 3)

    def both(x, a, b):
        y, u = R.lora_apply(batch, x, a, b, d["base"], keep=True)
        return (y, u) + R.lora_backward(batch, x, d["dy"], u, a, b)

    asked = [d[n].clone().requires_grad_() for n in ("x", "a", "b")]
    got = both(*asked)
    assert not any(t.requires_grad for t in got)
    assert all(torch.equal(p, q) for p, q in zip(got, both(d["x"], d["a"], d["b"])))
