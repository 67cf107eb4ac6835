"""What the library remembers of a device belongs to that device: another one of the process may have more or fewer SMs."""
import glob
import os
import re

import rotational_w4a4_quantization_gb300 as rq

CSRC = os.path.join(os.path.dirname(rq.__file__), "csrc")


def test_whatever_is_remembered_is_by_device():
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for kind, name, dims in re.findall(r"\bstatic std::atomic<([^>]+)> (\w+)((?:\[\w+\])*);", text):
            # a bit for each device, or a place
            by_bit = kind == "uint64_t" and re.search(r"allow_smem\([^;]*\b%s\)" % name, text)
            assert by_bit or dims.startswith("[kMaxDevices]"), (os.path.basename(path), kind, name + dims)
            found += 1
    assert found >= 6
