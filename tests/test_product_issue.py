"""The lane that issues tensor-core products commits them: a commit covers the issuing
thread's operations only, so that a commit by another lane completes at once, with
products still in flight.  Read from the sources: on the GPU nothing would show it but
an expired wait with products under way."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_13_gb300", "csrc")


def lanes(text, call):
    """First arguments of a file's calls, names taken for what they were set to."""
    found = set()
    for x in re.findall(call + r"\(\s*([^,]+?),", text):
        if x.startswith("uint32_t"):
            continue   # its definition
        found |= set(re.findall(r"const uint32_t %s = ([^;]+);" % re.escape(x), text)) or {x}
    names = {"(threadIdx.x & 31) == 0": "lane == 0"}
    return {names.get(x, x) for x in found}


@pytest.mark.parametrize("name", ["sv_attn_tc_kernel.cuh", "sv_row_tiles_tc.cuh",
                                  "sv_attn_weights_tc.cu"])
def test_products_are_committed_by_the_lane_that_issues_them(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    if name == "sv_row_tiles_tc.cuh":   # the load warp has a `lead` of its own
        text = text.replace("const uint32_t lead = lane == 0;", "", 1)
    issue = lanes(text, "mma_ss") | lanes(text, "mma_ts")
    assert len(issue) == 1 and lanes(text, "mma_commit") == issue


def test_every_kernel_with_products_is_looked_at():
    users = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*"))
             if re.search(r"mma_commit\(\s*lead", open(p).read())}
    assert users == {"sv_attn_tc_kernel.cuh", "sv_row_tiles_tc.cuh", "sv_attn_weights_tc.cu"}
