"""dlo_op_* calls may run in several host threads at once: what they write on the
host has to be their own (a local, a thread's) or synchronised.  Read from the
sources, since a lost increment of a shared counter shows nowhere else."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "layerwise_weight_offload_slot_gb300", "csrc")


@pytest.mark.parametrize("name", ["train_ops.cpp", "context.cpp"])
def test_the_entries_have_no_plain_counter_in_common(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    shared = re.findall(r"^(?:static )?(?:unsigned |signed )?(?:char|short|int|long|long long|size_t|u?int\d+_t|float|double|bool) \w+ *(?:=[^;(]*)?;", text, re.M)
    assert shared == []
