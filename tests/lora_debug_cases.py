"""Waits that gave up in the adapters' kernels, planted on the host, and who is told
of them: in a process of its own that loads the debug build (AFD_LIBRARY).  Called
by tests/test_lora_debug_gpu.py; prints one JSON line."""
import json
import os
import sys
from concurrent.futures import ThreadPoolExecutor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from combine_peer_slot_gb300 import afd as A  # noqa: E402


def told(stream):
    return [A.afd_lora_poll_status(stream.cuda_stream), A.afd_lora_poll_status(stream.cuda_stream)]


def case(site):
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    plant = lambda: A.afd_debug_plant(None, site)
    told(a), told(b)
    out = {"before": told(a) + told(b), "planted": plant()}
    out["first"], out["other_stream"] = told(a), told(b)
    with ThreadPoolExecutor(1) as ex:
        out["other_thread"] = ex.submit(told, a).result()
        plant(), plant()
        out["again"] = ex.submit(told, a).result() + told(a) + told(b)
    out["mx4"] = A.afd_mx4_poll_status(a.cuda_stream)
    return out


if __name__ == "__main__":
    A.lib()
    assert A.afd_debug_bounds(None)[0] == A.AFD_ERR_ARG, "not the debug build"
    torch.cuda.init()
    print(json.dumps([case(A.AFD_DBG_LORA_WAIT), case(A.AFD_DBG_LORA_WGRAD_WAIT)]))
