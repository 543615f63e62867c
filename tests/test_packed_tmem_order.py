"""The packed attention kernels by the reading of test_tmem_order: a fence behind every wait for tensor memory."""
import os

import pytest

from test_tmem_order import CSRC, unordered


@pytest.mark.parametrize("name", ["attention_packed.cu", "attention_packed_bwd.cu"])
def test_a_fence_follows_every_wait_for_tensor_memory(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    # what reads tensor memory behind a function's name
    text = text.replace("put_chunk(", "store_row (").replace("put_rows<", "store_row <")
    assert text.count("tc_fence_after()") > 5
    assert unordered(text) == []


def test_no_call_shares_plain_state():
    import test_op_calls_share_nothing as t
    t.test_the_entries_have_no_plain_counter_in_common("packed_ops.cpp")
