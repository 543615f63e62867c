"""Tensor memory handed from one thread to another: whoever waited on an mbarrier
for it runs tcgen05.fence::after_thread_sync before its next access, else nothing
orders that access behind what the barrier stands for.  A missing fence shows
as wrong numbers once in a long while, if at all, so the sources are read:
within a kernel, in the order of the text, no tensor memory access may follow a
wait without the fence between them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "layerwise_weight_offload_slot_gb300", "csrc")

EVENT = re.compile(r"(?P<wait>\b(?:mbar_wait|warp_wait|full)\()"
                   r"|(?P<fence>\btc_fence_after\()"
                   r"|(?P<access>\b(?:tmem_ld_\w+|tmem_st_\w+|tc_mma_\w+|mma_scores|mma_accumulate|store_row)\b)")


def unordered(text):
    """Lines with an access that follows a wait without a fence."""
    text = re.sub(r"//[^\n]*", "", text)
    found = []
    for body in re.finditer(r"__global__.*?\n}\n", text, re.S):
        waited = False
        for m in EVENT.finditer(body.group()):
            if m["access"] and waited:
                found.append(text.count("\n", 0, body.start() + m.start()) + 1)
            elif not m["access"]:
                waited = m["wait"] is not None
    return found


@pytest.mark.parametrize("name", ["attention_bwd.cu", "attention_tc.cu"])
def test_a_fence_follows_every_wait_for_tensor_memory(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert text.count("tc_fence_after()") > 5
    assert unordered(text) == []


def test_the_reading_finds_a_missing_fence():
    good = "__global__ void k() {\n    mbar_wait(b, 0);\n    tc_fence_after();\n    tmem_st_32x32b_x16(t, w);\n}\n"
    assert unordered(good) == []
    assert unordered(good.replace("    tc_fence_after();\n", "    // tc_fence_after();\n")) == [4]
