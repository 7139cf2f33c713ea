"""Refusals of the expert load, the routing gradient and the adapters: every
bad argument is answered before the device is touched (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B
from combine_peer_slot_gb300 import runtime as R

P = 0x10000  # an aligned address that is never dereferenced
WRAP = 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if B.needs_build():
        B.build()
    return A.lib()


BALANCE = dict(logits=P, ld=64, n_tokens=4, logits_dtype=A.AFD_DTYPE_F32, ids=P, num_experts=64, topk=6,
               score=A.AFD_SCORE_SOFTMAX, seq_offsets=P, n_seqs=2, loss=P, counts=P)


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(num_experts=0), dict(num_experts=257, ld=257), dict(topk=0), dict(topk=17), dict(ld=63),
    dict(topk=7, num_experts=6), dict(logits_dtype=2), dict(score=2), dict(n_seqs=0), dict(n_seqs=65536),
    dict(seq_offsets=0), dict(seq_offsets=P + 2), dict(logits=0), dict(ids=0), dict(loss=0), dict(counts=0),
    dict(logits=P + 2), dict(ids=P + 1), dict(loss=P + 2), dict(counts=P + 2)])
def test_balance_refuses(bad):
    assert A.afd_balance_loss(**{**BALANCE, **bad}) == A.AFD_ERR_ARG


def test_balance_workspace():
    assert A.afd_balance_workspace(512, 64, 4) == 0
    n = A.afd_balance_workspace(13312, 64, 4)
    assert n > 0 and n % (4 * 64 * 8) == 0
    for bad in ((-1, 64, 1), (4, 0, 1), (4, 257, 1), (4, 64, 0), (4, 64, 65536)):
        assert A.afd_balance_workspace(*bad) == -1
    big = {**BALANCE, "n_tokens": 13312, "n_seqs": 4}
    assert A.afd_balance_loss(**big, workspace=P, workspace_bytes=n - 1) == A.AFD_ERR_CAPACITY
    assert A.afd_balance_loss(**big, workspace=0, workspace_bytes=n) == A.AFD_ERR_ARG
    assert A.afd_balance_loss(**big, workspace=P + 64, workspace_bytes=n) == A.AFD_ERR_ARG


BACK = dict(logits=P, ld=64, n_tokens=4, logits_dtype=A.AFD_DTYPE_F32, ids=P, num_experts=64, topk=6,
            score=A.AFD_SCORE_SOFTMAX, renorm=True, routed_scaling=1.0, d_weights=P, seq_offsets=0, n_seqs=1, counts=P,
            d_loss=P, d_logits=P, ldd=64)


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(num_experts=0), dict(num_experts=257, ld=257, ldd=257), dict(topk=0), dict(topk=17),
    dict(ld=63), dict(ldd=63), dict(logits_dtype=3), dict(score=-1), dict(n_seqs=2), dict(counts=0), dict(d_loss=0),
    dict(logits=0), dict(d_logits=0), dict(ids=0), dict(logits=P + 1), dict(d_logits=P + 2), dict(d_weights=P + 2),
    dict(ids=P + 2), dict(counts=P + 1), dict(d_loss=P + 2)])
def test_route_backward_refuses(bad):
    assert A.afd_route_backward(**{**BACK, **bad}) == A.AFD_ERR_ARG


def test_plan_refuses():
    n = A.afd_lora_plan_bytes(100, 8)
    assert n > 0
    for bad in ((-1, 8), (2 ** 24 + 1, 8), (4, 0), (4, 1025)):
        assert A.afd_lora_plan_bytes(*bad) == -1
    ok = dict(ids=P, n_tokens=100, n_adapters=8, plan=P, plan_bytes=n)
    for bad, rc in ((dict(ids=0), A.AFD_ERR_ARG), (dict(ids=P + 2), A.AFD_ERR_ARG), (dict(plan=0), A.AFD_ERR_ARG),
                    (dict(plan=P + 16), A.AFD_ERR_ARG), (dict(plan_bytes=n - 1), A.AFD_ERR_CAPACITY),
                    (dict(n_tokens=-1), A.AFD_ERR_ARG), (dict(n_adapters=1025), A.AFD_ERR_ARG)):
        assert A.afd_lora_plan(**{**ok, **bad}) == rc, bad


APPLY = dict(plan=P, n_tokens=4, n_adapters=2, x=P, ldx=64, x_dtype=A.AFD_DTYPE_BF16, K=64, a=P, b=P, rank=8, M=32,
             scale=P, base=P, ldb=32, y_dtype=A.AFD_DTYPE_F32, out=P + 4096, ldo=32, u=P)


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(n_tokens=2 ** 24 + 1), dict(n_adapters=0), dict(n_adapters=1025), dict(K=0, ldx=0),
    dict(K=65537, ldx=65537), dict(M=0), dict(M=65537, ldb=65537, ldo=65537), dict(rank=0), dict(rank=129),
    dict(x_dtype=2), dict(y_dtype=-1), dict(ldx=63), dict(ldb=31), dict(ldo=31), dict(plan=0), dict(plan=P + 16),
    dict(x=0), dict(a=0), dict(b=0), dict(out=0), dict(x=P + 1), dict(a=P + 1), dict(b=P + 1), dict(out=P + 2),
    dict(base=P + 2), dict(scale=P + 2), dict(u=P + 2), dict(base=P, out=P, ldb=40), dict(out=P)])
def test_apply_refuses(bad):
    assert A.afd_lora_apply(**{**APPLY, **bad}) == A.AFD_ERR_ARG


GRAD = dict(plan=P, n_tokens=4, n_adapters=2, x=P, ldx=64, x_dtype=A.AFD_DTYPE_BF16, K=64, dy=P, ldy=32,
            y_dtype=A.AFD_DTYPE_F32, M=32, u=P, a=P, b=P, rank=8, scale=P, d_base=P, ldb=64, dx=P + 4096, ldd=64, da=P,
            db=P, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(n_adapters=1025), dict(K=0, ldx=0), dict(M=0), dict(rank=129), dict(x_dtype=2),
    dict(y_dtype=2), dict(ldx=63), dict(ldy=31), dict(ldd=63), dict(ldb=63), dict(plan=0), dict(x=0), dict(dy=0),
    dict(u=0), dict(a=0), dict(b=0), dict(dx=0), dict(da=0), dict(db=0), dict(workspace=0), dict(workspace=P + 64),
    dict(x=P + 1), dict(dy=P + 2), dict(u=P + 2), dict(da=P + 8), dict(db=P + 4), dict(dx=P + 1), dict(d_base=P + 1),
    dict(scale=P + 2), dict(d_base=P, dx=P, ldb=72), dict(dx=P)])
def test_backward_refuses(bad):
    assert A.afd_lora_backward(**{**GRAD, **bad}) == A.AFD_ERR_ARG


def test_backward_workspace():
    n = A.afd_lora_backward_workspace(2000, 2, 64, 32, 8, A.AFD_DTYPE_BF16, A.AFD_DTYPE_F32)
    assert n > 0 and n % 256 == 0
    for bad in ((-1, 8, 64, 32, 8, 0, 0), (4, 0, 64, 32, 8, 0, 0), (4, 8, 0, 32, 8, 0, 0), (4, 8, 64, 65537, 8, 0, 0),
                (4, 8, 64, 32, 129, 0, 0), (4, 8, 64, 32, 8, 2, 0), (4, 8, 64, 32, 8, 0, -1)):
        assert A.afd_lora_backward_workspace(*bad) == -1
    assert A.afd_lora_backward(**{**GRAD, "n_tokens": 2000, "workspace_bytes": n - 1}) == A.AFD_ERR_CAPACITY


def test_no_rows_is_no_work():
    assert A.afd_route_backward(**{**BACK, "n_tokens": 0, "logits": 0, "d_logits": 0}) == A.AFD_OK
    assert A.afd_lora_apply(**{**APPLY, "n_tokens": 0, "x": 0, "out": 0, "plan": 0}) == A.AFD_OK


# ---- what the torch wrappers refuse before the library is called ------------------
def refused(code, fn, *a, **kw):
    with pytest.raises(A.AfdError) as e:
        fn(*a, **kw)
    assert e.value.code == code


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


I, F, BF = torch.int32, torch.float32, torch.bfloat16


def test_gate_wrappers():
    l, ids = meta(4, 64), meta(4, 6, dtype=I)
    refused(A.AFD_ERR_NOT_DEVICE, R.balance_loss, l, ids)
    refused(A.AFD_ERR_NOT_DEVICE, R.route_backward, l, ids)
    for bad in (dict(logits=meta(4, 64, dtype=torch.float64)), dict(logits=meta(4, 257)), dict(logits=meta(64)),
                dict(logits=meta(WRAP + 4, 64), ids=meta(WRAP + 4, 6, dtype=I)), dict(ids=meta(5, 6, dtype=I)),
                dict(ids=meta(4, 6, dtype=torch.int64)), dict(ids=meta(4, 17, dtype=I)), dict(ids=meta(4, 0, dtype=I)),
                dict(ids=None), dict(score="max"), dict(seq_offsets=meta(1, dtype=I)), dict(seq_offsets=meta(3)),
                dict(logits=meta(64, 4).t())):
        refused(A.AFD_ERR_ARG, R.balance_loss, **{**dict(logits=l, ids=ids), **bad})
    refused(A.AFD_ERR_ARG, R.route_backward, l, None, d_weights=meta(4, 6))
    refused(A.AFD_ERR_ARG, R.route_backward, l, ids, counts=meta(1, 64, dtype=I))


def test_lora_wrappers():
    refused(A.AFD_ERR_NOT_DEVICE, R.LoraBatch, meta(4, dtype=I), 3)
    for ids, n in ((meta(4), 3), (meta(4, dtype=I), 0), (meta(4, dtype=I), 1025), (meta(4, dtype=I), WRAP + 3),
                   (meta(2 ** 24 + 1, dtype=I), 3), (meta(8, dtype=I)[::2], 3), (meta(2, 2, dtype=I), 3)):
        refused(A.AFD_ERR_ARG, R.LoraBatch, ids, n)
    batch = R.LoraBatch.__new__(R.LoraBatch)
    batch.plan, batch.rows, batch.adapters = meta(4096, dtype=torch.uint8), 4, 3
    ok = dict(batch=batch, x=meta(4, 64, dtype=BF), a=meta(3, 8, 64, dtype=BF), b=meta(3, 8, 32, dtype=BF),
              base=meta(4, 32))
    refused(A.AFD_ERR_NOT_DEVICE, R.lora_apply, **ok)
    for bad in (dict(x=meta(5, 64, dtype=BF)), dict(x=meta(4, 64, dtype=torch.float16)), dict(a=meta(3, 8, 64)),
                dict(a=meta(2, 8, 64, dtype=BF)), dict(b=meta(3, 9, 32, dtype=BF)), dict(a=meta(3, 129, 64, dtype=BF)),
                dict(a=meta(3, 8, WRAP + 64, dtype=BF)), dict(b=meta(3, 8, 65537, dtype=BF)),
                dict(x=meta(64, 4, dtype=BF).t())):
        refused(A.AFD_ERR_ARG, R.lora_apply, **{**ok, **bad})
    refused(A.AFD_ERR_NOT_DEVICE, R.lora_backward, batch, ok["x"], meta(4, 32), meta(4, 8), ok["a"], ok["b"])
    refused(A.AFD_ERR_ARG, R.lora_backward, batch, ok["x"], meta(4, 33), meta(4, 8), ok["a"], ok["b"])
