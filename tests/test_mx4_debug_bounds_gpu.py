"""The output rows of the MXFP4 products are checked in the debug build as those
of the other engines are (tests/mx4_debug_bounds_cases.py, in a process of its
own).  Needs an sm_103a GPU."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from combine_peer_slot_gb300 import afd as A
from combine_peer_slot_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def results():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if B.needs_build(debug=True):
        B.build(debug=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "mx4_debug_bounds_cases.py")], cwd=ROOT,
                       env=dict(os.environ, AFD_LIBRARY=B.LIB_DBG), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("name", ["narrow", "wide", "grouped"])
def test_output_rows_are_checked(results, name):
    r = results[name]
    assert r["step"] == A.AFD_OK and r["bounds"] == A.AFD_OK
    assert r["planted_step"] == A.AFD_ERR_BOUNDS
    code, site, index, limit = r["planted"]
    assert (code, site, limit) == (A.AFD_ERR_BOUNDS, A.AFD_DBG_GEMM_OUT, 0) and index >= 0
    assert r["after_step"] == A.AFD_OK and r["after_bounds"] == A.AFD_OK and r["same"]


def test_an_error_is_told_to_every_caller(results):
    once = [A.AFD_ERR_TIMEOUT, A.AFD_OK]
    r = results["status"]
    assert r["before"] == [A.AFD_OK] * 4
    assert r["first"] == r["other_stream"] == r["other_thread"] == r["new_stream"] == once
    assert r["again"] == once * 3
