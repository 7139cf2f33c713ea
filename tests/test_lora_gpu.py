"""afd_lora_plan, afd_lora_apply and afd_lora_backward against plain 64-bit
forms.  Tolerances count steps: an fp32 sum of the tensor cores may cut where
it should round, 2 U a step of sixteen terms; u in two bf16 parts (bf16 out)
is within 2^-17 of itself, in three (fp32 out) within U; one rounding of the
output, half a step of its type."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from tests import tuning_reference as ref

U = ref.U
BF, F = torch.bfloat16, torch.float32
PARTS = {BF: 2.0 ** -17, F: U}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def make(T, K, M, rank, L, xt, yt, how, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if how == "mixed":
        ids = torch.randint(-1, L, (T,), generator=g, device="cuda")
    elif how == "runs":
        ids = torch.randint(-1, L, (8,), generator=g, device="cuda").repeat_interleave((T + 7) // 8)[:T]
    elif how == "one":
        ids = torch.full((T,), L - 1, device="cuda")
    else:
        ids = torch.full((T,), -1, device="cuda")
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(ids=ids.int(), x=r(T, K).to(xt), a=(r(L, rank, K) / math.sqrt(K)).to(BF),
                b=(r(L, rank, M) / math.sqrt(rank)).to(BF), scale=r(L), base=r(T, M).to(yt), dy=r(T, M).to(yt),
                d_base=r(T, K).to(xt))


def near(got, want, tol, what):
    assert got.shape == want.shape
    over = (got.double() - want).abs() - tol
    assert bool((over <= 0).all()), (what, float(over.max()), int((over > 0).sum()))


def check_apply(d, base="other", scale=True, out=None):
    T = d["x"].shape[0]
    batch = R.LoraBatch(d["ids"], d["a"].shape[0])
    s = d["scale"] if scale else None
    yt = d["base"].dtype
    want, u, eu, eo, size = ref.adapters(d["ids"], d["x"], d["a"], d["b"], s, None if base == "none" else d["base"])
    if base == "same":
        y = d["base"].clone()
        got, gu = R.lora_apply(batch, d["x"], d["a"], d["b"], y, scale=s, out=y, keep=True)
        assert got is y
    else:
        got, gu = R.lora_apply(batch, d["x"], d["a"], d["b"], d["base"] if base == "other" else None, scale=s,
                               out=out, out_dtype=yt, keep=True)
    assert got.dtype == yt and gu.dtype == F
    near(gu, u, eu, "u")
    tol = eo + PARTS[yt] * size
    near(got, want, tol + ref.HALF[yt] * (want.abs() + tol), "y")
    off = (d["ids"] < 0) | (d["ids"] >= d["a"].shape[0])
    if base != "none":
        assert torch.equal(got[off], d["base"][off])
    else:
        assert (got[off] == 0).all()
    assert (gu[off] == 0).all()
    return batch, got, gu


def check_backward(d, batch, u, base="other", scale=True, dx=None):
    s = d["scale"] if scale else None
    xt, to = d["x"].dtype, dx
    dx, da, db, eo, size, ea, eb = ref.adapter_grads(d["ids"], d["x"], d["dy"], u, d["a"], d["b"], s,
                                                     None if base == "none" else d["d_base"])
    if base == "same":
        t = d["d_base"].clone()
        gx, ga, gb = R.lora_backward(batch, d["x"], d["dy"], u, d["a"], d["b"], d_base=t, scale=s, dx=t)
    else:
        gx, ga, gb = R.lora_backward(batch, d["x"], d["dy"], u, d["a"], d["b"],
                                     d_base=d["d_base"] if base == "other" else None, scale=s, dx=to)
    tol = eo + PARTS[xt] * size
    near(gx, dx, tol + ref.HALF[xt] * (dx.abs() + tol), "dx")
    near(ga, da, ea + U * (da.abs() + ea), "da")
    near(gb, db, eb + U * (db.abs() + eb), "db")
    return gx, ga, gb


SIZES = [(1, 64, 64, 8, 1), (1, 2048, 2816, 16, 8), (5, 16, 24, 1, 3), (17, 40, 56, 13, 4), (33, 100, 60, 16, 5),
         (64, 33, 17, 7, 2), (200, 256, 512, 32, 7), (329, 512, 704, 16, 64), (1024, 72, 64, 4, 2),
         (1025, 128, 64, 8, 3), (1500, 200, 136, 40, 6), (2100, 64, 1000, 64, 1), (1300, 96, 72, 100, 4),
         (1100, 48, 40, 128, 2), (3000, 136, 60, 9, 300), (90, 1, 1, 1, 1000), (4000, 61, 1030, 24, 2),
         (50, 3000, 24, 33, 3), (1200, 24, 4100, 17, 5),
         (1030, 520, 264, 64, 3), (2600, 72, 72, 33, 9), (5000, 128, 200, 48, 40)]


@pytest.mark.parametrize("T,K,M,rank,L", SIZES)
@pytest.mark.parametrize("xt,yt", [(BF, BF), (BF, F), (F, F), (F, BF)])
def test_sizes(T, K, M, rank, L, xt, yt):
    d = make(T, K, M, rank, L, xt, yt, "runs" if T % 2 else "mixed", T + K)
    batch, _, u = check_apply(d)
    check_backward(d, batch, u)


@pytest.mark.parametrize("how", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("base", ["other", "same", "none"])
@pytest.mark.parametrize("T", [40, 1600])
def test_batches(how, base, T):
    d = make(T, 128, 192, 16, 6, BF, BF, how, T)
    batch, _, u = check_apply(d, base, scale=base != "none")
    _, da, db = check_backward(d, batch, u, base, scale=base != "none")
    seen = set(d["ids"].tolist())
    for l in range(6):
        assert bool((da[l] == 0).all()) == (l not in seen) == bool((db[l] == 0).all())


def test_ids_out_of_range():
    d = make(100, 64, 64, 8, 4, BF, BF, "mixed", 1)
    d["ids"][::7] = 4
    d["ids"][1::7] = -2 ** 31
    d["ids"][2::7] = 2 ** 31 - 1
    batch, _, u = check_apply(d)
    check_backward(d, batch, u)


@pytest.mark.parametrize("xt,yt", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("T", [30, 1100])
def test_pitches(xt, yt, T):
    """Rows of a wider matrix, aligned and not; nothing beside them is written."""
    for pitch, first in ((208, 8), (201, 1), (204, 4)):
        d = make(T, 160, 96, 16, 3, xt, yt, "mixed", pitch)
        wide = lambda t: torch.full((t.shape[0], pitch), 7.0, dtype=t.dtype, device="cuda")
        for n in ("x", "base", "dy", "d_base"):
            w = wide(d[n])
            v = w[:, first:first + d[n].shape[1]]
            v.copy_(d[n])
            d[n] = v
        o = wide(d["base"])
        batch, _, u = check_apply(d, out=o[:, first:first + 96])
        assert (o[:, :first] == 7).all() and (o[:, first + 96:] == 7).all()
        o = wide(d["d_base"])
        check_backward(d, batch, u, dx=o[:, first:first + 160])
        assert (o[:, :first] == 7).all() and (o[:, first + 160:] == 7).all()


@pytest.mark.parametrize("xt,yt", [(BF, BF), (BF, F), (F, F), (F, BF)])
@pytest.mark.parametrize("T,rank", [(30, 16), (1100, 16), (1100, 48), (1100, 100)])
def test_ragged_columns(xt, yt, T, rank):
    """Columns that end inside a word, 8 and 16 bytes, from rows that begin at
    any element; nothing beside the outputs' rows is written."""
    for K, M, pitch, first in ((161, 97, 203, 3), (162, 98, 206, 2), (164, 100, 208, 4), (67, 257, 265, 5)):
        d = make(T, K, M, rank, 3, xt, yt, "mixed", 11)
        for n in ("x", "base", "dy", "d_base"):
            v = torch.full((T, pitch), math.nan, dtype=d[n].dtype, device="cuda")[:, first:first + d[n].shape[1]]
            v.copy_(d[n])
            d[n] = v
        o = torch.full((T, pitch), 7.0, dtype=yt, device="cuda")
        batch, _, u = check_apply(d, out=o[:, first:first + M])
        assert (o[:, :first] == 7).all() and (o[:, first + M:] == 7).all()
        o = torch.full((T, pitch), 7.0, dtype=xt, device="cuda")
        check_backward(d, batch, u, dx=o[:, first:first + K])
        assert (o[:, :first] == 7).all() and (o[:, first + K:] == 7).all()


@pytest.mark.parametrize("T", [48, 1300])
@pytest.mark.parametrize("xt", [BF, F])
def test_not_finite_rows(T, xt):
    """A row's NaN or infinity reaches that row and its adapter's gradients only."""
    d = make(T, 96, 64, 16, 4, xt, xt, "mixed", 8)
    d["ids"][:4] = torch.tensor([-1, 1, 2, 1], device="cuda").int()
    clean = make(T, 96, 64, 16, 4, xt, xt, "mixed", 8)
    clean["ids"] = d["ids"]
    d["x"][0] = math.nan   # no adapter
    d["x"][1, 5] = math.nan
    d["x"][2, 7] = math.inf
    batch = R.LoraBatch(d["ids"], 4)
    y, u = R.lora_apply(batch, d["x"], d["a"], d["b"], d["base"], scale=d["scale"], keep=True)
    y0, u0 = R.lora_apply(batch, clean["x"], d["a"], d["b"], d["base"], scale=d["scale"], keep=True)
    rest = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[rest], y0[rest]) and torch.equal(u[rest], u0[rest])
    assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[2]).any()
    dx, da, db = R.lora_backward(batch, d["x"], d["dy"], u0, d["a"], d["b"], d_base=d["d_base"], scale=d["scale"])
    assert torch.isfinite(dx).all() and torch.isfinite(db).all()
    assert torch.isfinite(da[[0, 3]]).all()
    assert not torch.isfinite(da[1, :, 5]).any() and not torch.isfinite(da[2, :, 7]).any()
    assert torch.isfinite(da[1, :, 6:]).all()


def test_largest_values():
    """fp32 rows near the type's largest value, and subnormal ones, keep their bits."""
    T, K = 20, 32
    x = torch.zeros(T, K, device="cuda")
    x[torch.arange(T), torch.arange(T)] = torch.tensor([3.4028234e38, -3.4e38, 1e-40, 1.0000001, 16777215.0] * 4, device="cuda")
    a = torch.eye(K, device="cuda").unsqueeze(0).to(BF).contiguous()
    batch = R.LoraBatch(torch.zeros(T, dtype=torch.int32, device="cuda"), 1)
    y, u = R.lora_apply(batch, x, a, a, out_dtype=F, keep=True)
    ok = x.abs() > 1e-37  # (parts of subnormal values are under the products' range)
    assert torch.equal(u[ok], x[ok]) and torch.equal(y[ok], x[ok])
    assert (u[~ok].abs() < 1e-37).all()


def test_no_rows():
    z = lambda *s, t=BF: torch.zeros(*s, dtype=t, device="cuda")
    batch = R.LoraBatch(z(0, t=torch.int32), 3)
    a, b = z(3, 4, 16), z(3, 4, 24)
    assert R.lora_apply(batch, z(0, 16), a, b, z(0, 24)).shape == (0, 24)
    da, db = torch.ones(3, 4, 16, device="cuda"), torch.ones(3, 4, 24, device="cuda")
    dx, _, _ = R.lora_backward(batch, z(0, 16), z(0, 24), z(0, 4, t=F), a, b, da=da, db=db)
    assert dx.shape == (0, 16) and (da == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T", [100, 2000])
def test_repeats_streams_and_graphs(T):
    """Equal bits from call to call, from two streams at a time with one plan, and from a graph with new rows and ids."""
    d = make(T, 256, 320, 16, 5, BF, BF, "mixed", 4)
    batch = R.LoraBatch(d["ids"], 5)

    def both(bt):
        y, u = R.lora_apply(bt, d["x"], d["a"], d["b"], d["base"], scale=d["scale"], keep=True)
        return (y, u) + R.lora_backward(bt, d["x"], d["dy"], u, d["a"], d["b"], d_base=d["d_base"], scale=d["scale"])

    first = both(batch)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s in sides:
            with torch.cuda.stream(s):
                got.append(both(batch))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in got for p, q in zip(o, first))
    assert A.afd_lora_poll_status(torch.cuda.current_stream().cuda_stream) == A.AFD_OK
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inner = R.LoraBatch(d["ids"], 5)
        held = both(inner)
    other = make(T, 256, 320, 16, 5, BF, BF, "runs", 5)
    for n in ("ids", "x", "dy", "base"):
        d[n].copy_(other[n])
    graph.replay()
    again = both(R.LoraBatch(d["ids"], 5))
    assert all(torch.equal(p, q) for p, q in zip(held, again)) and not torch.equal(again[0], first[0])


@pytest.mark.parametrize("T,rank", [(40, 16), (1200, 8), (1200, 48)])
def test_offsets_over_32_bits(T, rank):
    """Rows whose elements lie past 2^31 elements and 2^32 bytes from the first."""
    K, M = 64, 96
    d = make(T, K, M, rank, 3, BF, BF, "mixed", 9)
    pitch = (5 * 2 ** 29) // T // 8 * 8
    big = torch.empty(T * pitch, dtype=BF, device="cuda").view(T, pitch)
    for n, first in (("x", 0), ("base", 64), ("dy", 160), ("d_base", 256)):
        v = big[:, first:first + d[n].shape[1]]
        v.copy_(d[n])
        d[n] = v
    batch, _, u = check_apply(d, out=big[:, 320:320 + M])
    check_backward(d, batch, u, dx=big[:, 416:416 + K])


def test_many_rows_and_adapters():
    """200000 rows of all 1024 adapters: every tile, piece and block of the plan."""
    d = make(200000, 16, 24, 4, 1024, BF, BF, "mixed", 13)
    batch, y, u = check_apply(d)
    check_backward(d, batch, u)


def test_gradients_against_differences():
    """da, db and dx against central differences of the 64-bit form."""
    d = make(70, 24, 40, 5, 3, F, F, "mixed", 6)
    batch = R.LoraBatch(d["ids"], 3)
    _, u = R.lora_apply(batch, d["x"], d["a"], d["b"], d["base"], scale=d["scale"], keep=True)
    dx, da, db = R.lora_backward(batch, d["x"], d["dy"], u, d["a"], d["b"], scale=d["scale"])
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def value(x, a, b):
        return float((ref.adapters(d["ids"], x, a, b, d["scale"], None)[0] * d["dy"].double()).sum())

    x, a, b = d["x"].double(), d["a"].double(), d["b"].double()
    h = 1e-4
    for which, grad in ((0, dx), (1, da), (2, db)):
        args = [x, a, b]
        way = torch.randn(args[which].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + h * way, args[which] - h * way
        want = (value(*up) - value(*down)) / (2 * h)  # (exact for products of the first degree)
        got = float((grad.double() * way).sum())
        size = float((grad.double() * way).abs().sum())
        assert abs(got - want) <= 1e-5 * size, which
