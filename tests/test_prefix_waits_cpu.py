"""The second pass of shared-prefix attention may be resident long before the first has ended, and some of its warps
then stand in a wait without a limit.  A limited wait of the others must not run out meanwhile: it counts from the end
of the first pass."""
import os
import re

import rotational_w4a4_quantization_gb300 as rq

CSRC = os.path.join(os.path.dirname(rq.__file__), "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_a_wait_that_has_run_out_stands_behind_the_first_pass():
    text = source("tree_device.cuh")
    body = text[text.index("bool t_mbar_wait("):]
    body = body[:body.index("\n}\n")]
    late = body[body.index("if (clock64() > limit)"):]
    # past the limit: first the other pass's end and a new count, then, the next time, the error
    assert re.search(r"limit = \(clock64\(\) \+ kTreeWaitLimit\) & -2ll;", body)
    assert (late.index("if (PASS && !(limit & 1))") < late.index("pass_wait()") < late.index("limit = (clock64() + kTreeWaitLimit) | 1ll")
            < late.index("continue") < late.index("atomicExch(err, 1)"))


def test_the_waits_of_warps_that_do_not_go_on_from_the_first_pass_know_of_it():
    """Few rows: the producer's, on the consumers; many: all but the softmax warps'."""
    few, many = source("attn_tree_mma.cuh"), source("attn_tree_tc.cuh")
    assert re.findall(r"\b(t_mbar_wait\S*)\(&s\.(\w+)", few) == [("t_mbar_wait<P::kPass>", "empty"), ("t_mbar_wait<false>", "full")]
    calls = re.findall(r"\bwarp_wait(\S*)\(&s\.", many)
    assert len(calls) == 8 and set(calls) == {"<P::kPass>"}
    softmax = many[many.index("warp >= 4 && warp < 4 + kSoftWarps"):]
    assert len(re.findall(r"\bt_mbar_wait<false>\(&s\.", softmax)) == len(re.findall(r"\bt_mbar_wait\S*\(&s\.", many)) == 4
