"""The first call of a process captured into a graph: nothing has to run before.  Each in a process of its own."""
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
from test_gpu_packed import KEEP, Packed, dlo, scratch
p = Packed(%s)
a = p.desc()
ws = [scratch(f(a)) for f in (dlo.dlo_attention_packed_fwd_workspace_bytes, dlo.dlo_attention_packed_bwd_workspace_bytes)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    p.forward(ws[0])
    p.backward(ws[1])
torch.cuda.synchronize()
assert bool((p.o == KEEP).all()) and all(bool((t == KEEP).all()) for t in p.g)       # captured only
graph.replay()
torch.cuda.synchronize()
p.check(p.reference(), grads=True)
print("checked")
"""


@pytest.mark.parametrize("case", ["4, 2, 64, [130, 0, 300], None, 1", "2, 2, 72, [100, 31], None, 0", "16, 16, 72, [300] * 12, None, 0",
                                  "2, 1, 128, [200, 5], None, 1", "2, 2, 128, [17, 0, 9], [5000, 10, 300], 1",
                                  "2, 2, 64, [2500], [100], 0"])
def test_captured(case):
    r = subprocess.run([sys.executable, "-c", PROGRAM % case], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["checked"], r.stderr[-2000:]
