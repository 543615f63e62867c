"""The documented environment switches reach the training ops (read once per process, so each setting has its own)."""
import os
import subprocess
import sys

import pytest

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.path[:0] = ["tests", "."]
import torch
from torch.profiler import ProfilerActivity, profile
from test_gpu_train import Problem
p = Problem(2, 16, 16, 72, 1024, 1024)        # 256 query tiles: more than one an SM
p.forward()
torch.cuda.synchronize()
for _ in range(2):                            # the first one of a process may come out empty
    with profile(activities=[ProfilerActivity.CUDA]) as t:
        p.forward()
        torch.cuda.synchronize()
p.check(p.reference())
print("\\n".join(e.name for e in t.events() if "attn_tc_kernel" in e.name))
"""


def two_per_sm(**env):
    env = {**{k: v for k, v in os.environ.items() if k != "DLO_ATTN_DUO"}, **env}
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    names = [x for x in r.stdout.splitlines() if "attn_tc_kernel<" in x]
    assert len(names) == 1, r.stdout
    # attn_tc_kernel<blocks, tail, two CTAs per SM, training>
    form = [x.replace("(bool)", "").strip() for x in names[0].split("attn_tc_kernel<")[1].split(">")[0].split(",")]
    assert len(form) == 4 and form[2] in ("true", "false", "1", "0")
    return form[2] in ("true", "1")


def test_attn_duo_holds_for_the_training_forward():
    assert two_per_sm()
    assert not two_per_sm(DLO_ATTN_DUO="0")
