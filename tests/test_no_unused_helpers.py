"""No helper of the device code is left without a caller."""
import glob
import os
import re
from collections import Counter

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_tp_gb300", "csrc")
DEFINITION = re.compile(r"__device__\s+(?:__forceinline__\s+|constexpr\s+)*[\w:<>*& ]+?\b(\w+)\s*\(")


def test_every_device_helper_has_a_caller():
    text = ""
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as fh:
            text += re.sub(r"//.*", "", fh.read())
    defined = Counter(DEFINITION.findall(text))  # overloads count
    assert len(defined) > 60
    unused = sorted(n for n in defined if len(re.findall(rf"\b{n}\b", text)) <= defined[n])
    assert not unused, unused
