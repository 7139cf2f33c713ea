"""A block's shared memory may be reached from its cluster only once it is known to
have started: in every kernel a cluster barrier stands before the first such access
(read from the sources; no GPU needed)."""
import os
import re

from combine_peer_slot_gb300 import build as B

CSRC = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "csrc")
REACH = re.compile(r"map_shared_rank|shared::cluster\.(?:s32|u32|b32|f32|b64)|fr_mapa\(")
MEET = re.compile(r"cluster\.sync\(\)|barrier\.cluster\.wait|cluster_sync\(\)")


def kernels():
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
        starts = [m.start() for m in re.finditer(r"__global__", text)]
        for a in starts:
            end = text.find("\n}\n", a)
            yield name, text[a:end]


def test_clusters_meet_before_they_reach():
    seen = 0
    for name, body in kernels():
        reach = REACH.search(body)
        if not reach:
            continue
        seen += 1
        meet = MEET.search(body)
        assert meet and meet.start() < reach.start(), (name, body[:120])
    assert seen >= 4
