"""Rules that every source of the library keeps, checked on the text."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_csa2_gb300", "csrc")


def test_no_multicast_copies():
    """bench.py runs the same kernels on several GPUs, and copies that one CTA
    sends to a whole cluster are for code that runs on a single one."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            copies = re.findall(r"cp\.async\.bulk[^;]*;", f.read())
        assert not [c for c in copies if "multicast" in c], name
