"""Packed attention where a CTA takes over many items: several times as many items as an SM
has room for, of unequal lengths, so that what is carried from one item to the next
(barriers' phases, slots of the rings, tensor memory columns, row statistics) is used.
Against the plain form in 64 bits of the packed operators' other tests, with its bounds."""
import numpy as np
import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

from test_gpu_packed import Packed, float32_by_default, scratch  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def lengths(seed, n, low, high):
    """n lengths of 0 and of low .. high, one whole number of tiles and one of a row among them."""
    rng = np.random.default_rng(seed)
    v = rng.integers(low, high + 1, n)
    v[rng.random(n) < 0.1] = 0
    v[n // 2], v[n // 3] = 256, 1
    return v.tolist()


@pytest.mark.parametrize("heads", [(16, 8), (12, 12), (20, 4)], ids=str)
@pytest.mark.parametrize("hd", [64, 72, 128])
def test_backward_keeps_its_bits_over_many_calls(hd, heads):
    """An arrival counted for another step, or a wait that misses a phase, shows up rarely: as other bits, or as the
    error word of a wait that ran out."""
    p = Packed(*heads, hd, lengths(1, 24, 100, 700), None, 1 if heads[0] == 16 else 0)
    p.forward()
    a = p.desc()
    ws = scratch(dlo.dlo_attention_packed_bwd_workspace_bytes(a))
    p.backward(ws)
    p.check(p.reference(), grads=True)
    keep = [t.clone() for t in p.g]
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        for t in p.g:
            t.fill_(1.0)
        p.backward(ws)
        for x, y in zip(keep, p.g):
            w = (heads[0] if y is p.g[0] else heads[1]) * hd
            differ += (x[:, :w] != y[:, :w])[p.qs[0]:p.qs[-1]].sum()
    assert int(differ.item()) == 0 and int(p.err.item()) == 0
