"""What no kernel of the library may hold, found in its sources."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rag_kv_cache_rerotate_gb300", "csrc")


def test_no_copy_is_multicast_to_a_cluster():
    # the kernels also run as ranks of several GPUs, where such a copy has no place
    found = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for asm in re.findall(r'"[^"]*cp\.async\.bulk[^"]*"', text):
            if "multicast" in asm:
                found.append((name, asm))
    assert not found, found
