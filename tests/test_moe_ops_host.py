"""Refusals of the routing choice and of the MXFP4 entry points: every bad
argument is answered before the device is touched (no GPU needed)."""
import pytest

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B

P = 0x10000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if B.needs_build():
        B.build()
    return A.lib()


SELECT = dict(logits=P, ld=64, n_tokens=4, logits_dtype=A.AFD_DTYPE_F32, bias=0, num_experts=64, topk=6,
              score=A.AFD_SCORE_SOFTMAX, n_groups=1, topk_groups=1, group_top=1, renorm=False,
              routed_scaling=1.0, ids=P, weights=P)


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(num_experts=0), dict(num_experts=257, ld=257), dict(topk=0), dict(topk=17),
    dict(topk=7, num_experts=6), dict(ld=63), dict(logits_dtype=2), dict(score=2), dict(n_groups=0),
    dict(n_groups=33), dict(n_groups=5), dict(n_groups=8, topk_groups=0), dict(n_groups=8, topk_groups=9),
    dict(group_top=0), dict(group_top=3), dict(n_groups=32, topk_groups=2), dict(logits=0), dict(ids=0),
    dict(weights=0), dict(logits=P + 2), dict(ids=P + 1), dict(weights=P + 2), dict(bias=P + 1)])
def test_select_refuses(bad):
    assert A.afd_route_select(**{**SELECT, **bad}) == A.AFD_ERR_ARG


def test_no_rows_is_no_work():
    assert A.afd_route_select(**{**SELECT, "n_tokens": 0, "logits": 0, "ids": 0, "weights": 0}) == A.AFD_OK
    assert A.afd_mx4_quantize(**{**QUANT, "n_rows": 0, "x_rows": 0, "x": 0, "codes": 0, "scales": 0}) == A.AFD_OK
    assert A.afd_mx4_dequantize(**{**DEQUANT, "n_rows": 0, "codes": 0, "scales": 0, "out": 0}) == A.AFD_OK
    assert A.afd_mx4_gemm(**{**GEMM, "n_rows": 0, "codes": 0, "scales": 0, "out": 0}) == A.AFD_OK
    assert A.afd_mx4_ffn(**{**FFN, "n_rows": 0, "codes": 0, "scales": 0, "out": 0, "workspace": 0,
                            "workspace_bytes": 0}) == A.AFD_OK


QUANT = dict(x=P, ldx=64, x_rows=4, cols=64, dtype=A.AFD_DTYPE_BF16, src_rows=0, topk=1, n_rows=4,
             scale_rule=A.AFD_MX4_SCALE_FLOOR, codes=P, scales=P)


@pytest.mark.parametrize("bad", [
    dict(cols=0, ldx=0), dict(cols=48), dict(cols=65568, ldx=65568), dict(ldx=32), dict(dtype=5), dict(x_rows=-1),
    dict(n_rows=-1), dict(n_rows=5), dict(topk=2), dict(topk=0), dict(scale_rule=2), dict(x=0), dict(codes=0),
    dict(scales=0), dict(x=P + 8), dict(codes=P + 4), dict(ldx=68), dict(src_rows=P + 2),
    dict(n_rows=2 ** 30 + 1, src_rows=P)])
def test_quantize_refuses(bad):
    assert A.afd_mx4_quantize(**{**QUANT, **bad}) == A.AFD_ERR_ARG


DEQUANT = dict(codes=P, scales=P, n_rows=4, cols=64, dtype=A.AFD_DTYPE_F32, out=P, ldo=64)


@pytest.mark.parametrize("bad", [dict(cols=16), dict(dtype=-1), dict(n_rows=-1), dict(ldo=63), dict(ldo=65),
                                 dict(codes=0), dict(scales=0), dict(out=0), dict(codes=P + 8), dict(out=P + 4)])
def test_dequantize_refuses(bad):
    assert A.afd_mx4_dequantize(**{**DEQUANT, **bad}) == A.AFD_ERR_ARG


def test_weight_bytes():
    # 128 x 128 blocks of 8192 code and 512 scale bytes, edges rounded up
    assert A.afd_mx4_weight_bytes(1, 128, 128, False) == 8704
    assert A.afd_mx4_weight_bytes(3, 136, 96, False) == 3 * 2 * 8704
    assert A.afd_mx4_weight_bytes(64, 2816, 2048, True) == 64 * 22 * 16 * 8704
    assert A.afd_mx4_weight_bytes(1, 16, 32, True) == 8704
    for bad in ((0, 128, 128, False), (257, 128, 128, False), (1, 0, 128, False), (1, 12, 128, False),
                (1, 24, 128, True), (1, 128, 48, False), (1, 65544, 128, False), (1, 128, 65568, False)):
        assert A.afd_mx4_weight_bytes(*bad) == 0, bad


def test_pack_weight_refuses():
    ok = dict(codes=P, scales=P, num_experts=2, M=128, K=128, swiglu=False, packed=P, packed_bytes=17408)
    for bad, rc in ((dict(M=12), A.AFD_ERR_ARG), (dict(packed_bytes=17407), A.AFD_ERR_CAPACITY),
                    (dict(codes=0), A.AFD_ERR_ARG), (dict(scales=0), A.AFD_ERR_ARG), (dict(packed=0), A.AFD_ERR_ARG),
                    (dict(packed=P + 64), A.AFD_ERR_ARG), (dict(codes=P + 8), A.AFD_ERR_ARG)):
        assert A.afd_mx4_pack_weight(**{**ok, **bad}) == rc, bad


GEMM = dict(codes=P, scales=P, n_rows=4, offsets=P, num_experts=2, weight=P, M=128, K=128, swiglu=False,
            out_dtype=A.AFD_DTYPE_BF16, out=P, ldo=128)


@pytest.mark.parametrize("bad", [
    dict(n_rows=-1), dict(n_rows=2 ** 30 + 1), dict(num_experts=0), dict(num_experts=257), dict(M=12), dict(K=40),
    dict(ldo=120), dict(ldo=132), dict(out_dtype=3), dict(codes=0), dict(scales=0), dict(offsets=0), dict(weight=0),
    dict(out=0), dict(codes=P + 8), dict(scales=P + 2), dict(weight=P + 64), dict(out=P + 8), dict(offsets=P + 2)])
def test_gemm_refuses(bad):
    assert A.afd_mx4_gemm(**{**GEMM, **bad}) == A.AFD_ERR_ARG


def test_gemm_workspace():
    assert A.afd_mx4_gemm_workspace(96, 2, 128) == 0        # 48 rows a group: nothing needed
    n = A.afd_mx4_gemm_workspace(400, 2, 320)
    assert n == (3 + 2) * 3 * 1024                          # token tiles x 128-column blocks of images
    for bad in ((-1, 2, 128), (4, 0, 128), (4, 257, 128), (4, 2, 48)):
        assert A.afd_mx4_gemm_workspace(*bad) == -1, bad
    big = {**GEMM, "n_rows": 400, "K": 320}
    assert A.afd_mx4_gemm(**{**big, "workspace": P, "workspace_bytes": n - 1}) == A.AFD_ERR_CAPACITY
    assert A.afd_mx4_gemm(**{**big, "workspace": 0, "workspace_bytes": n}) == A.AFD_ERR_ARG
    assert A.afd_mx4_gemm(**{**big, "workspace": P + 128, "workspace_bytes": n}) == A.AFD_ERR_ARG


def test_gemm_swiglu_is_bf16():
    assert A.afd_mx4_gemm(**{**GEMM, "swiglu": True, "out_dtype": A.AFD_DTYPE_F32}) == A.AFD_ERR_UNSUPPORTED


FFN = dict(codes=P, scales=P, n_rows=4, offsets=P, num_experts=2, w13=P, wd=P, hidden=128, inter=64,
           out_dtype=A.AFD_DTYPE_BF16, out=P, ldo=128, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("bad", [
    dict(n_rows=-1), dict(num_experts=0), dict(hidden=100), dict(inter=48), dict(inter=0), dict(out_dtype=9),
    dict(ldo=96), dict(ldo=130), dict(codes=0), dict(scales=0), dict(offsets=0), dict(w13=0), dict(wd=0),
    dict(out=0), dict(workspace=0), dict(workspace=P + 16), dict(w13=P + 32), dict(out=P + 4)])
def test_ffn_refuses(bad):
    assert A.afd_mx4_ffn(**{**FFN, **bad}) == A.AFD_ERR_ARG


def test_ffn_workspace():
    n = A.afd_mx4_ffn_workspace(100, 2, 128, 96)
    assert n > 0 and n % 256 == 0
    assert A.afd_mx4_ffn_workspace(0, 2, 128, 96) == 0
    for bad in ((-1, 2, 128, 96), (4, 2, 128, 40), (4, 0, 128, 96), (4, 257, 128, 96), (4, 2, 130, 96)):
        assert A.afd_mx4_ffn_workspace(*bad) == -1, bad
    assert A.afd_mx4_ffn(**{**FFN, "n_rows": 100, "inter": 96, "workspace_bytes": n - 1}) == A.AFD_ERR_CAPACITY


def test_mx4_configuration():
    ok = dict(num_peers=2, token_cap=64, hidden=256, num_experts=8, topk=2, inter=64, shared_inter=32,
              flags=A.AFD_CFG_MX4)
    assert A.afd_slot_layout(A.make_config(**ok)).window_bytes > 0
    for bad in (dict(hidden=264), dict(inter=48), dict(shared_inter=48), dict(gemm=A.AFD_GEMM_SIMT),
                dict(gemm=A.AFD_GEMM_TENSOR_1CTA), dict(act="f32", gemm=A.AFD_GEMM_SIMT)):
        with pytest.raises(A.AfdError) as e:
            A.afd_slot_layout(A.make_config(**{**ok, **bad}))
        assert e.value.code == A.AFD_ERR_UNSUPPORTED, bad
    with pytest.raises(A.AfdError) as e:
        A.afd_slot_layout(A.make_config(**{**ok, "flags": 16}))
    assert e.value.code == A.AFD_ERR_ARG
