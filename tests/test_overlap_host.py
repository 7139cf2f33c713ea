"""What the calls write may not share a byte with what they read (no GPU needed:
refused before the device is touched)."""
import random

import pytest

torch = pytest.importorskip("torch")

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B

P = 1 << 20  # addresses that are never dereferenced, far apart
FAR = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if B.needs_build():
        B.build()
    return A.lib()


def apply(**kw):
    base = dict(plan=10 * FAR, n_tokens=4, n_adapters=2, x=P, ldx=64, x_dtype=A.AFD_DTYPE_BF16, K=64, a=11 * FAR, b=12 * FAR,
                rank=8, M=32, scale=13 * FAR, base=14 * FAR, ldb=32, y_dtype=A.AFD_DTYPE_F32, out=15 * FAR, ldo=32,
                u=16 * FAR)
    return A.afd_lora_apply(**{**base, **kw})


def backward(**kw):
    base = dict(plan=10 * FAR, n_tokens=4, n_adapters=2, x=P, ldx=64, x_dtype=A.AFD_DTYPE_BF16, K=64, dy=2 * FAR, ldy=32,
                y_dtype=A.AFD_DTYPE_F32, M=32, u=16 * FAR, a=11 * FAR, b=12 * FAR, rank=8, scale=13 * FAR, d_base=14 * FAR,
                ldb=64, dx=15 * FAR, ldd=64, da=17 * FAR, db=18 * FAR, workspace=19 * FAR, workspace_bytes=1 << 20)
    return A.afd_lora_backward(**{**base, **kw})


def route(**kw):
    base = dict(logits=P, ld=64, n_tokens=4, logits_dtype=A.AFD_DTYPE_F32, ids=2 * FAR, num_experts=64, topk=6,
                score=A.AFD_SCORE_SOFTMAX, renorm=True, routed_scaling=1.0, d_weights=3 * FAR, seq_offsets=4 * FAR, n_seqs=2,
                counts=5 * FAR, d_loss=6 * FAR, d_logits=7 * FAR, ldd=64)
    return A.afd_route_backward(**{**base, **kw})


def balance(**kw):
    base = dict(logits=P, ld=64, n_tokens=4, logits_dtype=A.AFD_DTYPE_F32, ids=2 * FAR, num_experts=64, topk=6,
                score=A.AFD_SCORE_SOFTMAX, seq_offsets=3 * FAR, n_seqs=2, loss=4 * FAR, counts=5 * FAR)
    return A.afd_balance_loss(**{**base, **kw})


def taken(code):
    """past the arguments' checks: what is asked next is the device"""
    return code in (A.AFD_ERR_CUDA, A.AFD_ERR_NOT_DEVICE)


def test_apart():
    assert all(taken(f()) for f in (apply, backward, route, balance))
    assert taken(apply(out=14 * FAR)) and taken(backward(dx=14 * FAR)) and taken(route(d_logits=P))
    # columns of one buffer
    assert taken(apply(x=P, ldx=160, base=P + 128, ldb=80, out=P + 128, ldo=80))
    assert taken(route(logits=P, ld=128, d_logits=P + 256, ldd=128))


@pytest.mark.parametrize("call,bad", [
    (apply, dict(out=P)), (apply, dict(out=P + 8)), (apply, dict(out=P - 8)), (apply, dict(out=14 * FAR + 4)),
    (apply, dict(out=14 * FAR - 128)), (apply, dict(out=11 * FAR + 512)), (apply, dict(out=12 * FAR)),
    (apply, dict(out=10 * FAR)), (apply, dict(out=13 * FAR)), (apply, dict(u=P + 16)), (apply, dict(u=14 * FAR)),
    (apply, dict(u=15 * FAR + 16)), (apply, dict(u=11 * FAR)), (apply, dict(base=15 * FAR, u=15 * FAR)),
    (backward, dict(dx=P + 64)), (backward, dict(dx=2 * FAR)), (backward, dict(dx=14 * FAR + 2)), (backward, dict(da=P)),
    (backward, dict(db=16 * FAR)), (backward, dict(da=18 * FAR)), (backward, dict(workspace=15 * FAR)),
    (backward, dict(workspace=17 * FAR)), (backward, dict(workspace=P)), (backward, dict(dx=11 * FAR)),
    (route, dict(d_logits=P + 4)), (route, dict(d_logits=P, ldd=80)), (route, dict(d_logits=2 * FAR)),
    (route, dict(d_logits=3 * FAR)), (route, dict(d_logits=5 * FAR)), (route, dict(d_logits=6 * FAR)),
    (route, dict(d_logits=4 * FAR)), (balance, dict(loss=P)), (balance, dict(counts=2 * FAR)),
    (balance, dict(loss=5 * FAR)), (balance, dict(counts=3 * FAR))])
def test_overlaps_are_refused(call, bad):
    assert call(**bad) == A.AFD_ERR_ARG


def test_rows_against_their_bytes():
    """Rows of any two pitches at any distance: refused where a byte is shared, and only there."""
    rng = random.Random(3)
    seen = [0, 0]
    for _ in range(6000):
        T, K, M = rng.randint(1, 6), rng.randint(1, 12), rng.randint(1, 12)
        ldx = K + rng.choice((0, 0, rng.randint(0, 20)))
        ldo = M + rng.choice((0, 0, rng.randint(0, 20)))
        if rng.random() < 0.5:
            ldx = ldo = max(ldx, ldo)
        at = P + 2 * rng.randint(-80, 80)
        x = {P + 2 * (t * ldx + c) for t in range(T) for c in range(K)}
        meet = any(at + 2 * (t * ldo + c) in x for t in range(T) for c in range(M))
        code = apply(n_tokens=T, K=K, M=M, ldx=ldx, ldo=ldo, ldb=M, out=at, y_dtype=A.AFD_DTYPE_BF16)
        assert code == A.AFD_ERR_ARG if meet else taken(code), (T, K, M, ldx, ldo, at - P)
        seen[meet] += 1
    assert min(seen) > 500


def test_two_rows_too_many_to_walk():
    """Interleaved rows of one pitch are told apart at once, whatever their number."""
    big = dict(n_tokens=2 ** 24, K=64, M=32, y_dtype=A.AFD_DTYPE_BF16, plan=1 << 50, a=1 << 51, b=1 << 52, u=1 << 53, scale=0,
               base=0, ldx=128, ldo=128)
    assert taken(apply(out=P + 128, **big))
    assert apply(out=P + 126, **big) == A.AFD_ERR_ARG
    assert apply(out=P + 192 - 2, **{**big, "M": 34}) == A.AFD_ERR_ARG
