"""The join of tree attention is launched beside the kernel whose partials it reads, so
every path through it has to pass its wait."""
import os
import re

import rotational_w4a4_quantization_gb300 as rq

SOURCE = os.path.join(os.path.dirname(rq.__file__), "csrc", "tree_device.cuh")


def test_no_path_leaves_the_join_before_its_wait():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    body = text[text.index("attn_tree_join_kernel("):]
    before = body[:body.index("griddepcontrol.wait")]
    assert not re.search(r"\breturn\b", before)
    assert before.count("{") - before.count("}") == 1          # and the wait stands under no condition
