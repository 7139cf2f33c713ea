"""The FFN step with its experts in MXFP4 (AFD_CFG_MX4) against a 64-bit form
of the same step on the same bytes: rows, weights and SwiGLU rows coded by
the format's definition, products in fp64, the routing taken from the step.

The two sides' SwiGLU rows differ by the rounding to bf16 at most, rarely (a
value within 2^-16 of a bf16 midpoint), and a code moves only where such a
value also lies within 2^-8 of itself of one of the 7 midpoints of the e2m1
grid: under one value in 2000, by at most a third of its block's largest, so
under 1 % of the rows' norm and of the outputs'.  The output's own rounding to
bf16 adds 2^-8 at most."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import runtime as R
from combine_peer_slot_gb300 import workloads as W
from tests import gpu_parity as G
from tests import mx4_reference as ref

TOL = 0.01 + 2.0 ** -8


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    A.lib()


def coded(x):
    return ref.decode(*ref.encode(x))


def ffn64(xq, W13, Wd):
    """fp64 rows of one expert from coded rows and raw bf16 weights."""
    h = ref.swiglu(xq @ coded(W13).T).bfloat16()
    return coded(h) @ coded(Wd).T


def step64(run, layer, x, ids, w, with_shared=True):
    """[T, H] fp64: the weighted sum of the routed experts and the shared one."""
    wt = run.weights[layer]
    xq = coded(x)
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in range(run.w.num_experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            out[t] += w[t, j].double().unsqueeze(1) * ffn64(xq[t], wt["W13"][e], wt["Wd"][e])
    if with_shared and run.w.shared_inter:
        out += ffn64(xq, wt["W13s"], wt["Wds"])
    return out


def routing(run, T):
    k = run.w.topk
    ids = torch.from_numpy(G.ws_array(run, A.AFD_WS_IDS, T * k, np.int32).reshape(T, k).copy()).cuda()
    w = torch.from_numpy(G.ws_array(run, A.AFD_WS_WEIGHTS, T * k, np.float32).reshape(T, k).copy()).cuda()
    return ids, w


def close(got, want):
    err = float((got.double() - want).norm() / want.norm().clamp(min=1e-30))
    assert err <= TOL, err


def check_forward(w, layers=1, **kw):
    run = R.Runner(w, layers=layers, flags=A.AFD_CFG_MX4, **kw)
    for layer in range(layers):
        run.pack_all(layer)
        assert run.forward(layer) == 0
        outs = run.unpack_all()
        assert run.poll() == 0
        G.check_canaries(run)
        T = w.total_tokens
        if not T:
            continue
        ids, wts = routing(run, T)
        want = step64(run, layer, torch.cat([x for x, n in zip(run.x, w.seq_lens) if n]), ids, wts)
        close(torch.cat([o[:n] for o, n in zip(outs, w.seq_lens)]), want)
    run.close()


@pytest.mark.parametrize("lens", [[37, 91], [1, 0], [5, 5], [300, 450], [0, 0]])
def test_fanin(lens):
    """Few rows per expert and many, an empty peer, an empty fan-in."""
    check_forward(W.custom("fanin", seq_lens=lens), canary=True)


def test_no_shared_expert_and_layers():
    check_forward(W.custom("fanin", seq_lens=[64, 130], shared_inter=0, layers=2), layers=2)


@pytest.mark.parametrize("hidden,inter,shared", [(96, 32, 32), (288, 96, 160), (544, 352, 96)])
def test_odd_sizes(hidden, inter, shared):
    check_forward(W.custom("fanin", seq_lens=[77, 202], hidden=hidden, inter=inter, shared_inter=shared))


def test_v2lite_layer():
    check_forward(W.custom("v2lite_prefill", seq_lens=[9, 700]))


def test_stays_after_a_failed_step_and_takes_new_weights():
    w = W.custom("fanin", seq_lens=[20, 30])
    run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4, wait_timeout_ns=20_000_000)
    assert run.forward(0) == 0            # nothing packed: the bounded wait gives up
    assert run.poll() == A.AFD_ERR_TIMEOUT
    run.weights[0] = W.expert_weights(W.custom("fanin", seq_lens=[20, 30], seed=77), 0, "cuda")
    wt = run.weights[0]
    A.afd_set_layer(run.ctx, 0, run.Wg.data_ptr(), 0, wt["W13"].data_ptr(), wt["Wd"].data_ptr(),
                    wt["W13s"].data_ptr(), wt["Wds"].data_ptr())
    run.pack_all(0)
    assert run.forward(0) == 0
    outs = run.unpack_all()
    assert run.poll() == 0
    ids, wts = routing(run, 50)
    close(torch.cat([o[:n] for o, n in zip(outs, w.seq_lens)]), step64(run, 0, torch.cat(run.x), ids, wts))
    run.close()


def test_grouped_form():
    """The Attention side routes: every row's expert output comes back."""
    w = W.custom("fanin", seq_lens=[60, 111])
    run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4, max_total_tokens=w.total_tokens,
                   )
    run.prepare_grouped(seed=3)
    if max(run.g_n) > w.token_cap:
        run.close()
        w = W.custom("fanin", seq_lens=[60, 111], token_cap=64 * -(-max(run.g_n) // 64))
        run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4, max_total_tokens=w.total_tokens)
        run.prepare_grouped(seed=3)
    run.pack_grouped_all(0)
    assert run.forward_grouped(0) == 0
    ys, ss = run.unpack_grouped_all()
    assert run.poll() == 0
    wt = run.weights[0]
    for p, n in enumerate(w.seq_lens):
        want, at = [], 0
        for e, c in enumerate(run.g_list[p]):
            if c:
                want.append(ffn64(coded(run.g_rows[p][at:at + c]), wt["W13"][e], wt["Wd"][e]))
            at += c
        close(ys[p][:run.g_n[p]], torch.cat(want))
        close(ss[p][:n], ffn64(coded(run.x[p]), wt["W13s"], wt["Wds"]))
    run.close()


@pytest.mark.parametrize("graph", [False, True])
def test_work_item_loop(graph):
    """Steps whose layer and counts the device takes from the headers, eager
    and replayed: the same outputs as the host-described step."""
    w = W.custom("fanin", seq_lens=[37, 91], layers=3)
    run = R.Runner(w, layers=3, ring_depth=2, flags=A.AFD_CFG_MX4, max_total_tokens=w.total_tokens)
    g = None
    if graph:
        rc, g, kernels = A.afd_serve_graph_create(run.ctx, [0, 1], 1)
        assert rc == 0 and kernels > 0
    for stage, layer, counts in ((0, 2, [37, 91]), (1, 0, [20, 50]), (0, 1, [0, 91]), (1, 2, [3, 0])):
        seqs = []
        for p, n in enumerate(counts):
            run.seq += 1
            assert A.afd_pack_slot(run.ctx, p, stage, layer, run.x[p].data_ptr() if n else 0, n, True, run.seq) == 0
            seqs.append(run.seq)
        assert (A.afd_serve_graph_launch(g) if graph else A.afd_ffn_serve(run.ctx, [0, 1], 1)) == 0
        for p, n in enumerate(counts):
            assert A.afd_unpack_split(run.ctx, p, stage, run.out[p].data_ptr() if n else 0, n, seqs[p]) == 0
        assert run.poll() == 0
        T = sum(counts)
        ids, wts = routing(run, T)
        x = torch.cat([run.x[p][:n] for p, n in enumerate(counts) if n])
        got = torch.cat([run.out[p][:n] for p, n in enumerate(counts) if n])
        close(got, step64(run, layer, x, ids, wts))
    if graph:
        A.afd_serve_graph_destroy(g)
    run.close()


def test_token_level_dispatch_to_two_ranks(monkeypatch):
    """The experts split over two FFN ranks, each with its block in MXFP4."""
    plain = A.make_config
    monkeypatch.setattr(A, "make_config", lambda *a, **k: plain(*a, **{**k, "flags": A.AFD_CFG_MX4}))
    w = W.custom("fanin", seq_lens=[37, 91])
    rs = R.RankSet(w, 2)
    rs.route()
    rs.dispatch_all()
    rs.serve_all()
    outs = rs.combine_all()
    assert rs.poll() == (0, 0)
    for p, n in enumerate(w.seq_lens):
        xq = coded(rs.x[p])
        wt = rs.weights[0]
        want = ffn64(xq, wt["W13s"], wt["Wds"])
        for e in range(w.num_experts):
            t, j = (rs.ids[p][:n] == e).nonzero(as_tuple=True)
            if t.numel():
                want[t] += rs.wts[p][t, j].double().unsqueeze(1) * ffn64(xq[t], wt["W13"][e], wt["Wd"][e])
        # the ranks' outputs travel in bf16: another 2^-8 of each term
        assert float((outs[p][:n].double() - want).norm() / want.norm()) <= TOL + 2.0 ** -8
    rs.close()


def test_weights_that_are_mxfp4_already_are_kept():
    """bf16 weights whose values are MXFP4 values code to themselves."""
    w = torch.randn(300, 256, device="cuda").bfloat16()
    once = R.mx4_dequantize(R.mx4_quantize(w), torch.bfloat16)
    again = R.mx4_dequantize(R.mx4_quantize(once), torch.bfloat16)
    assert torch.equal(once, again)
