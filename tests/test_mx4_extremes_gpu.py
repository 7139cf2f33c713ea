"""The largest rows, columns and tensors that the MXFP4 calls take: 65536 in each
direction, and codes and outputs of over 2^31 elements (19 GB at most).  Rows
are copies of a few, scaled by powers of two, so that every output is known from a
few rows' 64-bit products.  A product's bound as in the tests of the product: 2^-24 of
the terms' magnitudes a term, and half a step of the output."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import mx4_reference as ref

GB = 1 << 30


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()
    yield
    assert A.afd_mx4_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK
    torch.cuda.empty_cache()


def room(gb):
    if torch.cuda.mem_get_info()[0] < gb * GB:
        pytest.skip(f"{gb} GB wanted")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weight(M, K, seed, swiglu=False):
    """Random codes with scales that keep the sums near 1; the packed weight and
    the plain one (its 64-bit values are taken in slices)."""
    g = gen(seed)
    codes = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    e = 125 - round(math.log2(K) / 2)
    scales = torch.randint(e - 2, e + 1, (M, K // 32), generator=g, device="cuda").to(torch.uint8)
    return R.Mx4Weight(codes.view(1, M, -1), scales.view(1, M, -1), swiglu=swiglu), (codes, scales)


def products(xv, plain):
    """y = W x and the terms' magnitudes in 64 bits."""
    codes, scales = plain
    y = torch.empty(xv.shape[0], codes.shape[0], dtype=torch.float64, device="cuda")
    s = torch.empty_like(y)
    step = max(8, (1 << 26) // xv.shape[1])
    for i in range(0, codes.shape[0], step):
        w = ref.decode(codes[i:i + step], scales[i:i + step])
        y[:, i:i + step] = xv @ w.T
        s[:, i:i + step] = xv.abs() @ w.abs().T
    return y, s


@pytest.mark.parametrize("rows", [3, 130])
@pytest.mark.parametrize("M,K,swiglu", [(8, 65536, False), (65536, 32, False), (16, 65536, True), (65536, 32, True),
                                        (65528, 65536, False)])
def test_largest_sizes(rows, M, K, swiglu):
    room(20)
    x = R.mx4_quantize(torch.randn(rows, K, generator=gen(rows), device="cuda"))
    w, plain = weight(M, K, M + K, swiglu)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y, s = products(ref.decode(x.codes, x.scales), plain)
    for dt in (torch.bfloat16,) if swiglu else (torch.bfloat16, torch.float32):
        out = R.mx4_gemm(x, off, w, out_dtype=dt).double()
        if swiglu:
            want, up = ref.swiglu(y), y[:, M // 2:]
            dg, du = K * 2.0 ** -24 * s[:, :M // 2], K * 2.0 ** -24 * s[:, M // 2:]
            gate = y[:, :M // 2]
            bound = (2.0 ** -8 + 2.0 ** -21) * want.abs() + 1.1 * (up.abs() + du) * dg + (gate / (1 + torch.exp(-gate))).abs() * du
        else:
            want, bound = y, torch.finfo(dt).eps / 2 * y.abs() + K * 2.0 ** -24 * s
        assert float(((out - want).abs() - bound).max()) <= 1e-38


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_over_2_to_31(dtype):
    room(40)
    n, M, K = 33000, 65536, 32
    base = torch.randn(3, K, generator=gen(1), device="cuda").bfloat16()
    src = (torch.arange(n, device="cuda") % 3).int()
    x = R.mx4_quantize(base, src_rows=src)
    w, plain = weight(M, K, 2)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = R.mx4_gemm(x, off, w, out_dtype=dtype)
    few = R.mx4_gemm(R.mx4_quantize(base), torch.tensor([0, 3], dtype=torch.int32, device="cuda"), w, out_dtype=dtype)
    y, s = products(ref.decode(x.codes[:3], x.scales[:3]), plain)
    assert float(((few.double() - y).abs() - torch.finfo(dtype).eps / 2 * y.abs() - K * 2.0 ** -24 * s).max()) <= 0
    for i in range(0, n, 3000):  # (equal rows: equal sums, whatever the form)
        assert torch.equal(out[i:i + 3000].view(-1, 3, M), few.expand(1000, 3, M))


def test_codes_over_2_to_31():
    """Coding, its reverse and a product over rows whose codes pass 2^31 bytes."""
    room(60)
    n, K = 66000, 65536
    base = torch.randn(2, K, generator=gen(3), device="cuda").bfloat16()
    x = torch.empty(n, K, dtype=torch.bfloat16, device="cuda")
    power = torch.exp2((torch.arange(n // 2, device="cuda") % 5).float()).bfloat16()
    for i in range(0, n // 2, 3000):
        x[2 * i:2 * i + 6000].view(-1, 2, K).copy_(base * power[i:i + 3000].view(-1, 1, 1))
    q = R.mx4_quantize(x)
    del x
    two = R.mx4_quantize(base)
    for i in range(0, n, 6000):
        assert torch.equal(q.codes[i:i + 6000].view(-1, 2, K // 2), two.codes.expand(3000, 2, K // 2))
        want = two.scales.int() + (torch.arange(i // 2, i // 2 + 3000, device="cuda") % 5).view(-1, 1, 1)
        assert torch.equal(q.scales[i:i + 6000].view(-1, 2, K // 32).int(), want)
    back = R.mx4_dequantize(q, torch.bfloat16)
    first = R.mx4_dequantize(two, torch.bfloat16)
    for i in range(0, n // 2, 3000):
        assert torch.equal(back[2 * i:2 * i + 6000].view(-1, 2, K), first * power[i:i + 3000].view(-1, 1, 1))
    del back
    w, _ = weight(8, K, 4)
    out = R.mx4_gemm(q, torch.tensor([0, n], dtype=torch.int32, device="cuda"), w, out_dtype=torch.float32)
    few = R.mx4_gemm(two, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), w, out_dtype=torch.float32)
    # powers of two scale every term and every rounding alike
    assert torch.equal(out.view(-1, 2, 8), few * power.float().view(-1, 1, 1))


@pytest.mark.parametrize("T,E", [(3_000_000, 2), (40_000_000, 1)])
def test_many_rows_to_route(T, E):
    room(10)
    logits = torch.randn(T, E, generator=gen(5), device="cuda")
    ids, w = R.route_select(logits, 1, score="sigmoid")
    want = logits.argmax(1, keepdim=True).int()
    assert torch.equal(ids, want)
    s = torch.sigmoid(logits.double().gather(1, want.long()))
    assert float((w.double() / s - 1).abs().max()) <= 8 * 2.0 ** -24
