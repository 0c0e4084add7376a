"""Cluster barriers of the .aligned form are a whole warp's instructions: the sources reach them through cluster_sync(), which
brings the warp together first."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bound_weight_gb300", "csrc")


def test_aligned_cluster_barriers_follow_a_warp_barrier():
    found = []
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                text = f.read()
            for at in re.finditer(r'asm volatile\("barrier\.cluster\.arrive[^;"]*\.aligned', text):
                before = text[:at.start()].rstrip().splitlines()[-1].strip()
                found.append((name, before))
    assert found and all(before == "__syncwarp();" for _, before in found), found
