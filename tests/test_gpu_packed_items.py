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


SMS = 152


def items(lens, heads, rows=128):
    return sum(-(-n // rows) for n in lens) * heads


SELF = lengths(2, 40, 30, 700)
OTHER = lengths(3, 40, 1, 600)           # keys of another packing, some sequences without any
MANY = [
    # H, G, hd, q lengths, k lengths, causal block
    (16, 8, 64, SELF, None, 1), (16, 8, 72, SELF, None, 1), (16, 8, 128, SELF, None, 1),
    (12, 12, 64, SELF, None, 0), (12, 12, 80, SELF, None, 0), (12, 12, 104, SELF, None, 0),
    (16, 8, 64, SELF, OTHER, 1), (16, 8, 72, SELF, OTHER, 1), (16, 8, 128, SELF, OTHER, 1),
    (16, 16, 64, SELF, OTHER, 0), (16, 16, 72, SELF, OTHER, 0), (16, 16, 128, SELF, OTHER, 0),
    (30, 6, 64, SELF, None, 100), (30, 6, 72, SELF, None, 100), (30, 6, 128, SELF, None, 100),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "%dx%dx%d-%s-%d" % (*c[:3], "cross" if c[4] else "self", c[5]))
def test_many_unequal_items(case):
    H, G, hd, ql, kl, cb = case
    # some three or more for every CTA that an SM has room for (forward: two up to head dim 80)
    assert items(ql, H) >= 4 * SMS and items(kl or ql, G) >= 3 * SMS
    assert items([n * (H // G) for n in ql], G) >= (4 if hd <= 80 else 3) * SMS
    p = Packed(H, G, hd, ql, kl, cb, lead=3, slack=5)
    ref = p.reference()
    p.forward()
    p.check(ref)
    p.backward()
    p.check(ref, grads=True)


@pytest.mark.parametrize("cb", [0, 1, 64])
@pytest.mark.parametrize("shape", [(8, 8, 64, 200, 4000), (8, 8, 72, 200, 4000), (4, 4, 128, 300, 9000), (16, 4, 64, 60, 9000),
                                   (8, 4, 64, 100, 9000), (20, 4, 128, 60, 4000), (16, 4, 64, 100, 4000)], ids=str)
def test_runs_of_keys_over_several_query_tiles(shape, cb):
    """Few queries over long keys: a CTA is a run of keys with an item for every query tile, and the rows' parts are
    joined.  The last shape has too many query tiles for that: CTAs of a query tile each."""
    H, G, hd, nq, nk = shape
    rng = np.random.default_rng(nk)
    ql, kl = (rng.integers(n - n // 2, n + n // 2, 6).tolist() for n in (nq, nk))
    kl[1], ql[4] = 0, 0
    p = Packed(H, G, hd, ql, kl, cb, lead=2, slack=1)
    split = dlo.dlo_attention_packed_fwd_workspace_bytes(p.desc()) > 2 * H * p.rq * hd * 4        # two parts a row or more
    assert split == (shape != (16, 4, 64, 100, 4000))
    ref = p.reference()
    p.forward()
    p.check(ref)
    first = [p.o.clone(), p.lse.clone()]
    for _ in range(50):
        p.forward()
    assert torch.equal(first[0], p.o) and torch.equal(first[1], p.lse)
    p.backward()
    p.check(ref, grads=True)
