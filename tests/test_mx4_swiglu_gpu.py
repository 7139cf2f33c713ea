"""The rounding of the SwiGLU rows.  Where the fp32 sums of gate and up are
exact, silu(gate) * up is left with its own fp32 arithmetic before the one
rounding to bf16, in units of 2^-24 of the value: the exponential 2 (it is
within one ulp), 1 + e 1, the division 1, the product 1: 5, taken as 5.1 for
their products.  Results under 2^-126 lose up to half of fp32's smallest step at
the division and the product; a reciprocal of 1 + e under 2^-126 may be zero,
which |gate| 2^-126 |up| bounds."""
import math

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
    yield
    assert A.afd_mx4_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK


def exact_sums(rows, I, K, seed):
    """Rows and weights whose products' sums are exact in fp32: every term is a
    multiple of 2^-8 (codes 2^-2, scales 2^-2 and 2^-4) and the sums stay under
    36 K 2^-1 < 2^11, 19 bits in all."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def draw(n, lo, hi):
        codes = torch.randint(0, 256, (n, K // 2), generator=g, device="cuda").to(torch.uint8)
        return codes, torch.randint(lo, hi + 1, (n, K // 32), generator=g, device="cuda").to(torch.uint8)

    return draw(rows, 125, 127), draw(2 * I, 123, 126)


@pytest.mark.parametrize("rows", [40, 2000])  # the narrow and the wide form
def test_rows_are_rounded_once(rows):
    I, K = 512, 64
    (xc, xs), (wc, ws) = exact_sums(rows, I, K, rows)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    weight = R.Mx4Weight(wc.view(1, 2 * I, -1), ws.view(1, 2 * I, -1), swiglu=True)
    out = R.mx4_gemm(R.Mx4(xc, xs), off, weight).double()
    y = ref.decode(xc, xs) @ ref.decode(wc, ws).T
    assert torch.equal(y.float().double(), y) and float(y.abs().max()) > 90
    want = ref.swiglu(y)
    _, ex = torch.frexp(want)
    half = torch.exp2((ex - 9).clamp(min=-134).double())  # half a bf16 step: 8 significant bits
    up = y[:, I:].abs()
    bound = half + 5.1 * 2.0 ** -24 * want.abs() + (up + 1) * 2.0 ** -150 + y[:, :I].abs() * up * 2.0 ** -126
    over = (out - want).abs() - bound
    assert float(over.max()) <= 0, (int((over > 0).sum()), over.numel())


@pytest.mark.parametrize("rows", [5, 100])  # the narrow and the wide form
def test_sums_that_overflow(rows):
    """Gates of +inf, -inf and the largest finite ones times up of every kind: as
    the formula in fp32 steps on the same sums (inf u; NaN for -inf, 0 times inf)."""
    K, gates, ups = 32, (6.0, -6.0, 1.0, -1.0, 0.0), (6.0, -6.0, 0.0, 0.5)
    pairs = [(g, s, u, t) for g in gates for s in (252, 130, 126, 4) for u in ups for t in (252, 127, 2)]
    pairs += pairs[:-len(pairs) % 8]
    I = len(pairs)
    code = {v: c for c, v in enumerate(ref.VALUES)}
    code.update({-v: c + 8 for v, c in list(code.items()) if v})
    codes = torch.zeros(1, 2 * I, K // 2, dtype=torch.uint8)
    scales = torch.full((1, 2 * I, 1), 127, dtype=torch.uint8)
    for i, (g, s, u, t) in enumerate(pairs):
        codes[0, i, 0], scales[0, i, 0] = code[g], s
        codes[0, I + i, 0], scales[0, I + i, 0] = code[u], t
    x = torch.zeros(rows, K // 2, dtype=torch.uint8)
    x[:, 0] = code[4.0]
    x = R.Mx4(x.cuda(), torch.full((rows, 1), 125, dtype=torch.uint8, device="cuda"))  # rows of 1, 0, 0 ..
    x.scales[1::2] = 252                                                              # and of 4 * 2^125
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    codes, scales = codes.cuda(), scales.cuda()
    y = R.mx4_gemm(x, off, R.Mx4Weight(codes, scales), out_dtype=torch.float32)
    g, u = y.chunk(2, -1)
    assert all(bool((g == v).any()) and bool((u == v).any()) for v in (math.inf, -math.inf))
    want = (g / (1 + torch.exp(-g)) * u).bfloat16().float()
    out = R.mx4_gemm(x, off, R.Mx4Weight(codes, scales, swiglu=True)).float()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(torch.isinf(out)[fine], torch.isinf(want)[fine])
    fin = fine & ~torch.isinf(want)
    assert torch.equal(out[fine & torch.isinf(want)], want[fine & torch.isinf(want)])
    err = (out[fin].double() - want[fin].double()).abs()
    assert bool((err <= 2.0 ** -8 * 1.01 * want[fin].double().abs() + (g[fin].abs().double() + 1) * u[fin].abs().double() * 2.0 ** -126).all())
