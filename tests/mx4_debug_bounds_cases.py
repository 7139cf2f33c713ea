"""MXFP4 steps against the bounds-checking debug build, in a process of its own
that loads that build (AFD_LIBRARY).  Called by tests/test_mx4_debug_bounds_gpu.py;
prints one JSON line.  Status: a planted error of a product without a context is told
once to every thread and stream that polls.  Clean steps: no check fails.  Planted: every check of the
products' output rows fails on valid rows (the bound is taken as 0, nothing is
stored), the step reports it, and a clean step gives the first one's bits."""
import json
import os
import sys
from concurrent.futures import ThreadPoolExecutor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from combine_peer_slot_gb300 import afd as A  # noqa: E402
from combine_peer_slot_gb300 import runtime as R  # noqa: E402
from combine_peer_slot_gb300 import workloads as W  # noqa: E402


def step(run, grouped):
    if grouped:
        run.pack_grouped_all(0)
        assert run.forward_grouped(0) == A.AFD_OK
    else:
        run.pack_all(0)
        assert run.forward(0) == A.AFD_OK
    torch.cuda.synchronize()


def bits(run, grouped):
    if grouped:
        ys, ss = run.unpack_grouped_all()
        return [t.clone() for t in ys + ss]
    return [t.clone() for t in run.unpack_all()]


def case(lens, grouped):
    w = W.custom("fanin", seq_lens=lens, token_cap=2048)
    run = R.Runner(w, layers=1, flags=A.AFD_CFG_MX4, max_total_tokens=w.total_tokens)
    if grouped:
        run.prepare_grouped(seed=5)
    step(run, grouped)
    first = bits(run, grouped)
    out = {"step": run.poll(), "bounds": A.afd_debug_bounds(run.ctx)[0]}
    assert A.afd_debug_plant(run.ctx, A.AFD_DBG_GEMM_OUT) == A.AFD_OK
    step(run, grouped)
    out["planted_step"] = run.poll()
    rec = A.afd_debug_bounds(run.ctx)
    out["planted"] = [int(v) for v in rec]
    assert A.afd_debug_plant(run.ctx, 0) == A.AFD_OK
    step(run, grouped)
    again = bits(run, grouped)
    out["after_step"], out["after_bounds"] = run.poll(), A.afd_debug_bounds(run.ctx)[0]
    out["same"] = all(torch.equal(a, b) for a, b in zip(first, again))
    run.close()
    return out


def told(stream):
    return [A.afd_mx4_poll_status(stream.cuda_stream), A.afd_mx4_poll_status(stream.cuda_stream)]


def status():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    out = {"before": told(a) + told(b)}
    assert A.afd_debug_plant(None, A.AFD_DBG_MX4_WAIT) == A.AFD_OK
    out["first"], out["other_stream"] = told(a), told(b)
    with ThreadPoolExecutor(1) as ex:
        out["other_thread"] = ex.submit(told, a).result()
        assert A.afd_debug_plant(None, A.AFD_DBG_MX4_WAIT) == A.AFD_OK
        assert A.afd_debug_plant(None, A.AFD_DBG_MX4_WAIT) == A.AFD_OK
        out["again"] = ex.submit(told, a).result() + told(a) + told(b)
    out["new_stream"] = told(torch.cuda.Stream())
    return out


def main():
    A.lib()
    assert A.afd_debug_bounds(None)[0] == A.AFD_ERR_ARG, "not the debug build"
    print(json.dumps({"status": status(), "narrow": case([37, 91], False), "wide": case([300, 450], False),
                      "grouped": case([60, 111], True)}))


if __name__ == "__main__":
    main()
