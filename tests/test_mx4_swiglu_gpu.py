"""The rounding of the SwiGLU rows.  Where the fp32 sums of gate and up are
exact, silu(gate) * up is left with its own fp32 arithmetic before the one
rounding to bf16, in units of 2^-24 of the value: the exponential 2 (it is
within one ulp), 1 + e 1, the division 1, the product 1: 5, taken as 5.1 for
their products.  Results under 2^-126 lose up to half of fp32's smallest step at
the division and the product; a reciprocal of 1 + e under 2^-126 may be zero,
which |gate| 2^-126 |up| bounds."""
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
