"""The numbers that the device status word reports: every wait of the kernels has its own."""
import glob
import os
import re
from collections import Counter

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_tp_gb300", "csrc")


def test_wait_sites_have_numbers_of_their_own():
    sites = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as fh:
            for name, n in re.findall(r"\b(kSite\w+)\s*=\s*(\d+)", fh.read()):
                assert name not in sites, f"{name} is defined twice"
                sites[name] = int(n)
    assert len(sites) >= 24
    twice = [n for n, k in Counter(sites.values()).items() if k > 1]
    assert not twice, {n: [s for s in sites if sites[s] == n] for n in twice}
