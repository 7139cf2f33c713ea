"""MXFP4 coding, the grouped product and the expert FFN against plain 64-bit
forms.

Coding is compared bit for bit.  A product's bound: every one of its K terms
is exact, the fp32 accumulation may lose 2^-24 of the running magnitude at
each term (at most S = sum |w| |x|), and the result is rounded once (half a
step: 2^-8 of a bf16 value, 2^-24 of an fp32 one).  SwiGLU adds its own
arithmetic: silu's slope is at most 1.1, the fast exponential and division
stay under 2^-19 of the value for |gate| <= 40."""
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


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def same_values(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])


# ---- coding --------------------------------------------------------------------
def check_coding(x, rule, **kw):
    q = R.mx4_quantize(x, rule=rule, **kw)
    src = x
    if "src_rows" in kw:
        i = kw["src_rows"].long() // kw.get("topk", 1)
        ok = (kw["src_rows"] >= 0) & (i < x.shape[0])
        src = torch.where(ok.unsqueeze(1), x[i.clamp(0, x.shape[0] - 1)], torch.zeros((), dtype=x.dtype, device="cuda"))
    codes, scales = ref.encode(src, rule)
    assert torch.equal(q.scales, scales)
    assert torch.equal(q.codes, codes)
    for dt in (torch.bfloat16, torch.float32):
        assert same_values(R.mx4_dequantize(q, dt).double(), ref.decode(codes, scales))
    return q


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2048), (3, 96), (37, 1024), (129, 1408), (1000, 160)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_quantize(rows, cols, dtype, rule):
    g = gen(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))
    check_coding(x.to(dtype), rule)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_quantize_borders(dtype, rule):
    """Every midpoint and value of the grid and their neighbours, at every
    exponent the type has, signed zeros, subnormals, zero blocks."""
    tiny = torch.finfo(dtype).eps / 2
    grid = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0],
                        dtype=torch.float64)
    vals = torch.cat([grid, -grid, grid * (1 + 2 * tiny), -grid * (1 - tiny)])  # 64 values
    tops = torch.tensor([4.0, 6.0, 6.0 * (1 + 2 * tiny), 7.9], dtype=torch.float64)
    rows = []
    for e in list(range(-149, -120)) + list(range(-6, 7)) + list(range(118, 126)):
        for top in tops:
            blk = vals.clone()
            blk[::32] = top
            rows.append(blk * 2.0 ** e)
    x = torch.stack(rows).clamp(-3.3e38, 3.3e38).to(dtype).cuda()
    x = torch.cat([x, torch.zeros(2, 64, dtype=dtype, device="cuda"), -torch.zeros(1, 64, dtype=dtype, device="cuda")])
    check_coding(x, rule)


def test_quantize_not_finite():
    """A block with a NaN or an infinity reads as NaN; the others do not."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(6, 128, generator=gen(1), device="cuda").to(dtype)
        x[0, 5] = math.nan
        x[1, 40] = math.inf
        x[2, 127] = -math.inf
        x[3] = math.nan
        q = check_coding(x, "floor")
        assert (q.scales == 255).sum() == 3 + 4


def test_quantize_gather_and_strides():
    g = gen(4)
    big = torch.randn(50, 512, generator=g, device="cuda").bfloat16()
    x = big[:, 64:64 + 288]
    src = torch.randint(0, 50 * 6, (311,), generator=g, device="cuda", dtype=torch.int32)
    src[3] = -1
    src[200] = 50 * 6        # one past the last position
    src[310] = 2 ** 31 - 1
    q = check_coding(x, "floor", src_rows=src, topk=6)
    assert (q.scales[3] == 0).all() and (q.codes[200] == 0).all()
    check_coding(x, "ceil")
    assert R.mx4_quantize(x[:0]).rows == 0
    none = R.mx4_quantize(x, src_rows=src[:0], topk=6)
    assert R.mx4_dequantize(none, torch.float32).shape == (0, 288)


# ---- grouped product -------------------------------------------------------------
def rows_and_weights(counts, M, K, seed, lead=0, behind=0, spread=1.0):
    g = gen(seed)
    n = sum(counts) + lead + behind
    scale = torch.exp(spread * torch.randn(n, 1, generator=g, device="cuda"))
    x = R.mx4_quantize(torch.randn(n, K, generator=g, device="cuda") * scale)
    E = len(counts)
    w = torch.randn(E, M, K, generator=g, device="cuda") / math.sqrt(K)
    w *= torch.exp(spread * torch.randn(E, M, 1, generator=g, device="cuda"))
    wq = R.mx4_quantize(w.view(E * M, K))
    codes, scales = wq.codes.view(E, M, K // 2), wq.scales.view(E, M, K // 32)
    off = torch.tensor([lead] + counts, device="cuda").cumsum(0).int()
    return x, off, codes, scales


def product_bound(y, s, K, dtype):
    return torch.finfo(dtype).eps / 2 * y.abs() + K * 2.0 ** -24 * s


def check_product(counts, M, K, dtype, swiglu=False, seed=0, lead=0, behind=0):
    x, off, codes, scales = rows_and_weights(counts, M, K, seed, lead, behind)
    w = R.Mx4Weight(codes, scales, swiglu=swiglu)
    cols = M // 2 if swiglu else M
    out = torch.full((x.rows, cols), 77.0, dtype=dtype, device="cuda")
    R.mx4_gemm(x, off, w, out_dtype=dtype, out=out)
    torch.cuda.synchronize()
    y, s = ref.grouped(ref.decode(x.codes, x.scales), off, ref.decode(codes, scales))
    if swiglu:
        h = ref.swiglu(y)
        dg = K * 2.0 ** -24 * s[:, :cols]
        du = K * 2.0 ** -24 * s[:, cols:]
        gate, up = y.chunk(2, -1)
        silu = gate / (1 + torch.exp(-gate))
        bound = (torch.finfo(dtype).eps / 2 + 2.0 ** -19) * h.abs() + 1.1 * (up.abs() + du) * dg + silu.abs() * du
        y = h
    else:
        bound = product_bound(y, s, K, dtype)
    n = x.rows
    inside = slice(lead, n - behind)
    err = (out.double() - y).abs()[inside] - bound[inside] - 1e-38
    assert not torch.isnan(err).any()
    assert err.numel() == 0 or float(err.max()) <= 0, (float(err.max()), (err > 0).nonzero()[:4])
    outside = torch.cat([out[:lead], out[n - behind:]])
    assert (outside == 77.0).all()
    return out


SHAPES = [
    ([1], 8, 32), ([1], 128, 256), ([5], 64, 64), ([16], 128, 128), ([17], 136, 96), ([64], 256, 512),
    ([65], 128, 1408), ([3, 0, 70, 1, 0, 0, 20, 9], 264, 320), ([0, 0, 4], 128, 2048), ([300], 128, 256),
    ([192], 256, 256), ([193], 384, 288), ([200, 1, 0, 577], 520, 736), ([0] * 255 + [3], 16, 64),
]


@pytest.mark.parametrize("counts,M,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(counts, M, K, dtype):
    check_product(counts, M, K, dtype, seed=len(counts) + M + K)


@pytest.mark.parametrize("counts,M,K", [(c, 2 * max(8, m // 16 * 8), k) for c, m, k in SHAPES])
def test_product_swiglu(counts, M, K):
    check_product(counts, M, K, torch.bfloat16, swiglu=True, seed=M + K)


@pytest.mark.parametrize("counts,M,K", [([2500, 3000], 2048, 1408), ([40] * 16, 2048, 1408), ([700, 1, 3300], 2816, 320)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_units_per_sm(counts, M, K, swiglu):
    """More output tiles than the GPU has SMs: every ring goes round many times."""
    check_product(counts, M, K, torch.bfloat16, swiglu=swiglu, seed=K)


@pytest.mark.parametrize("counts", [[7, 0, 30], [250, 400]])
def test_rows_outside_groups_keep_their_values(counts):
    for swiglu in (False, True):
        check_product(counts, 256, 320, torch.bfloat16, swiglu=swiglu, lead=5, behind=9)


def test_no_rows_in_any_group():
    check_product([0, 0, 0], 128, 256, torch.float32, behind=40)


def test_scales_per_block_and_far_apart():
    """Blocks whose scales differ by many powers of two, and NaN blocks that
    reach their own rows only."""
    g = gen(9)
    n, M, K = 100, 128, 512
    x = torch.randn(n, K, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-12, 13, (n, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)
    x[7, 100] = math.nan
    w = torch.randn(M, K, generator=g, device="cuda")
    w *= torch.exp2(torch.randint(-12, 13, (M, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)
    xq, wq = R.mx4_quantize(x), R.mx4_quantize(w)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    weight = R.Mx4Weight(wq.codes.view(1, M, -1), wq.scales.view(1, M, -1))
    out = R.mx4_gemm(xq, off, weight, out_dtype=torch.float32).double()
    assert torch.isnan(out[7]).all()
    y, s = ref.grouped(ref.decode(xq.codes, xq.scales), off, ref.decode(wq.codes, wq.scales).view(1, M, K))
    keep = torch.arange(n, device="cuda") != 7
    err = (out - y).abs() - product_bound(y, s, K, torch.float32)
    assert float(err[keep].max()) <= 0


def test_offsets_out_of_range_are_clamped():
    x, off, codes, scales = rows_and_weights([40, 60], 128, 256, 3)
    w = R.Mx4Weight(codes, scales)
    want = R.mx4_gemm(x, off, w)
    got = R.mx4_gemm(x, torch.tensor([-5, 40, 2 ** 30], dtype=torch.int32, device="cuda"), w)
    assert torch.equal(want, got)


def test_output_pitch():
    x, off, codes, scales = rows_and_weights([33, 60], 136, 256, 5)
    w = R.Mx4Weight(codes, scales)
    for dt in (torch.bfloat16, torch.float32):
        want = R.mx4_gemm(x, off, w, out_dtype=dt)
        big = torch.full((93, 200), 5.0, dtype=dt, device="cuda")
        R.mx4_gemm(x, off, w, out_dtype=dt, out=big[:, 16:152])
        assert torch.equal(big[:, 16:152], want)
        assert (big[:, :16] == 5.0).all() and (big[:, 152:] == 5.0).all()


# ---- expert FFN ------------------------------------------------------------------
def ffn_weights(E, hidden, inter, seed):
    g = gen(seed)
    w13 = R.mx4_quantize(torch.randn(E * 2 * inter, hidden, generator=g, device="cuda") / math.sqrt(hidden))
    wd = R.mx4_quantize(torch.randn(E * hidden, inter, generator=g, device="cuda") / math.sqrt(inter))
    return (R.Mx4Weight(w13.codes.view(E, 2 * inter, -1), w13.scales.view(E, 2 * inter, -1), swiglu=True),
            R.Mx4Weight(wd.codes.view(E, hidden, -1), wd.scales.view(E, hidden, -1)), w13, wd)


@pytest.mark.parametrize("counts,hidden,inter", [([1], 64, 32), ([5, 0, 1], 96, 160), ([90, 12], 256, 352),
                                                 ([0, 400, 200], 512, 96), ([6] * 32, 1024, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ffn_equals_its_parts(counts, hidden, inter, dtype):
    """Bit for bit the SwiGLU product, the coding of its rows and the down
    product, each of which is checked against the 64-bit form above."""
    g = gen(inter)
    n = sum(counts)
    x = R.mx4_quantize(torch.randn(n, hidden, generator=g, device="cuda").bfloat16())
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    w13, wd, _, _ = ffn_weights(len(counts), hidden, inter, 8)
    got = R.mx4_ffn(x, off, w13, wd, out_dtype=dtype)
    h = R.mx4_quantize(R.mx4_gemm(x, off, w13))
    want = R.mx4_gemm(h, off, wd, out_dtype=dtype)
    assert torch.equal(got, want)


def test_ffn_not_finite():
    """A NaN block of one row reaches that row's output only, as in the parts."""
    for counts in ([30, 5], [300, 250]):
        n = sum(counts)
        x = torch.randn(n, 256, generator=gen(2), device="cuda").bfloat16()
        x[7, 40] = math.nan
        x[n - 1, 255] = math.inf
        q = R.mx4_quantize(x)
        off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        w13, wd, _, _ = ffn_weights(2, 256, 96, 4)
        got = R.mx4_ffn(q, off, w13, wd)
        want = R.mx4_gemm(R.mx4_quantize(R.mx4_gemm(q, off, w13)), off, wd)
        assert same_values(got, want)
        bad = torch.isnan(got).all(1)
        assert bad[7] and bad[n - 1] and int(torch.isnan(got).any(1).sum()) == 2


@pytest.mark.parametrize("offsets", [[0, 400, 0, 400], [400, 0, 400, 0], [-7, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]])
def test_offsets_that_overlap_stay_in_bounds(offsets):
    """Not a valid call: its results mean nothing, but nothing outside its
    outputs and workspace is written and the next call is right."""
    w13, wd, _, _ = ffn_weights(3, 256, 96, 5)
    x = R.mx4_quantize(torch.randn(400, 256, generator=gen(6), device="cuda"))
    need = A.afd_mx4_ffn_workspace(400, 3, 256, 96)
    ws = torch.full((need + 65536,), 171, dtype=torch.uint8, device="cuda")
    out = torch.full((400 + 64, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    R.mx4_ffn(x, torch.tensor(offsets, device="cuda").int(), w13, wd, out=out[:400], workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 171).all() and (out[400:] == 3.0).all()
    off = torch.tensor([0, 100, 250, 400], device="cuda").int()
    want = R.mx4_gemm(R.mx4_quantize(R.mx4_gemm(x, off, w13)), off, wd)
    assert torch.equal(R.mx4_ffn(x, off, w13, wd, out=out[:400], workspace=ws[:need]), want)


# ---- together ----------------------------------------------------------------------
def test_gate_coding_experts_and_sum_together():
    """A layer as it is used: the gate's choice, positions by expert, the
    routed rows coded, the expert FFN, the weighted sum; against 64 bits.

    The two sides' h agree to 2^-8 (a bf16 rounding that falls the other way,
    rarely), and a code moves by one step only where h lies that near a
    midpoint of the grid: the share of values within 2^-8 of themselves of
    one of the 7 midpoints is under 5 %, and of those the rounding differs
    in under one in a hundred (the fp32 sums agree to 2^-16 of the 2^-8).  A
    step is at most a third of the block's largest, so the moved codes carry
    under sqrt(0.0005) * 0.33 < 1 % of h's norm, hence of y's."""
    g = gen(31)
    T, E, k, hidden, inter = 150, 24, 4, 256, 128
    xs = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    bias = 0.05 * torch.randn(E, generator=g, device="cuda")
    gate = dict(bias=bias, score="sigmoid", n_groups=4, topk_groups=2, group_top=2, renorm=True, routed_scaling=2.5)
    ids, w = R.route_select(logits, k, **gate)
    perm = ids.flatten().sort(stable=True).indices.int()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(ids.flatten(), minlength=E).cumsum(0)
    x = R.mx4_quantize(xs, src_rows=perm, topk=k)
    w13, wd, c13, cd = ffn_weights(E, hidden, inter, 6)
    y = R.mx4_ffn(x, off, w13, wd, out_dtype=torch.float32)
    out = torch.zeros(T, hidden, device="cuda", dtype=torch.float64)
    out.index_add_(0, perm.long() // k, y.double() * w.flatten()[perm.long()].double().unsqueeze(1))
    xv = ref.decode(*ref.encode(xs))
    a = ref.decode(c13.codes, c13.scales).view(E, 2 * inter, hidden)
    b = ref.decode(cd.codes, cd.scales).view(E, hidden, inter)
    rid, rw = ref.select(logits, k, **gate)
    assert torch.equal(ids.cpu(), rid)
    want = torch.zeros_like(out)
    for t in range(T):
        for j in range(k):
            e = int(rid[t, j])
            h = ref.swiglu((a[e] @ xv[t]).unsqueeze(0)).bfloat16()
            want[t] += float(rw[t, j]) * (b[e] @ ref.decode(*ref.encode(h))[0])
    assert float((out - want).norm() / want.norm()) <= 0.01


def test_streams_graphs_and_workspaces():
    """Two captured graphs with a workspace each, replayed in turn and on
    another stream, give the eager bits; inputs change between replays."""
    counts = [40, 0, 11, 90]
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    w13, wd, _, _ = ffn_weights(4, 256, 96, 3)
    xa = torch.randn(141, 256, generator=gen(1), device="cuda").bfloat16()
    xb = torch.randn(141, 256, generator=gen(2), device="cuda").bfloat16()
    want = {i: R.mx4_ffn(R.mx4_quantize(v), off, w13, wd) for i, v in (("a", xa), ("b", xb))}
    torch.cuda.synchronize()
    src = [xa.clone(), xb.clone()]
    graphs, outs, keep = [], [], []
    for s in src:
        ws = torch.empty(A.afd_mx4_ffn_workspace(141, 4, 256, 96), dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(R.mx4_ffn(R.mx4_quantize(s), off, w13, wd, workspace=ws))
        graphs.append(gr)
        keep.append(ws)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want["a"]) and torch.equal(outs[1], want["b"])
    src[0].copy_(xb)
    src[1].copy_(xa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want["b"]) and torch.equal(outs[1], want["a"])


def test_repeats_give_the_same_bits():
    x, off, codes, scales = rows_and_weights([70, 0, 300, 5], 512, 704, 12)
    w = R.Mx4Weight(codes, scales)
    first = R.mx4_gemm(x, off, w)
    for _ in range(5):
        assert torch.equal(R.mx4_gemm(x, off, w), first)


@pytest.mark.parametrize("K", [32, 128, 160, 256, 288, 384, 416, 512, 544, 768, 800, 1024, 1056])
@pytest.mark.parametrize("swiglu", [False, True])
def test_wide_rows_that_end_in_every_part_of_a_stage(K, swiglu):
    """Groups large enough for the wide form; the row's end in the first or
    the second half of a 512-column stage, or none of it in the second."""
    check_product([150, 230, 0, 90], 272, K, torch.bfloat16, swiglu=swiglu, seed=K)


@pytest.mark.parametrize("counts,K", [([100], 8192), ([70, 193], 4128), ([300, 5, 1000], 2080)])
def test_wide_few_tiles_of_long_rows(counts, K):
    """A token tile's scale image by several CTAs, in uneven shares."""
    check_product(counts, 128, K, torch.float32, seed=K)


def test_swiglu_at_the_ends_of_the_exponential():
    """Gates whose exponential overflows, vanishes or is nearly 1, up = 1: the
    exponential is off by (4 + 2 |g|) 2^-24, its sum and reciprocal by 3, and
    results of the reciprocal under 2^-126 are zero; then one rounding to bf16."""
    values = [s * m * 2.0 ** e for s in (1, -1) for m in (1.0, 1.5) for e in range(-20, 8)]
    I, K = len(values), 32
    assert I % 8 == 0
    w = torch.zeros(2 * I, K, device="cuda")
    w[:I, 0] = torch.tensor(values, device="cuda")
    w[I:, 0] = 1.0
    wq = R.mx4_quantize(w)
    weight = R.Mx4Weight(wq.codes.view(1, 2 * I, -1), wq.scales.view(1, 2 * I, -1), swiglu=True)
    for rows in (3, 100):
        x = torch.zeros(rows, K, device="cuda")
        x[:, 0] = 1.0
        off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        out = R.mx4_gemm(R.mx4_quantize(x), off, weight).double()
        g = torch.tensor(values, device="cuda", dtype=torch.float64)
        want = g / (1 + torch.exp(-g))
        bound = (2.0 ** -8 + (12 + 2 * g.abs()) * 2.0 ** -24) * want.abs() + (g.abs() + 1) * 2.0 ** -126
        assert not torch.isnan(out).any()
        assert ((out - want).abs() <= bound).all()
