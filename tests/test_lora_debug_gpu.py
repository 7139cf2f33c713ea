"""A wait of the adapters' kernels that gave up is told once to every thread and
stream that polls (tests/lora_debug_cases.py, in a process of its own)."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_an_error_is_told_to_every_caller():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if B.needs_build(debug=True):
        B.build(debug=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "lora_debug_cases.py")], cwd=ROOT,
                       env=dict(os.environ, AFD_LIBRARY=B.LIB_DBG), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    once = [A.AFD_ERR_TIMEOUT, A.AFD_OK]
    cases = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(cases) == 2
    for c in cases:
        assert c["planted"] == A.AFD_OK and c["before"] == [A.AFD_OK] * 4
        assert c["first"] == c["other_stream"] == c["other_thread"] == once
        assert c["again"] == once * 3 and c["mx4"] == A.AFD_OK


def test_release_build_plants_nothing():
    if B.needs_build():
        B.build()
    A.lib()
    for site in (A.AFD_DBG_LORA_WAIT, A.AFD_DBG_LORA_WGRAD_WAIT):
        assert A.afd_debug_plant(None, site) == A.AFD_ERR_UNSUPPORTED
