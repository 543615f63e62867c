"""Rows that get no part of an attention problem -- behind the lengths, or with nothing
to see -- are zeros (lse -inf) whatever a tile's other rows hold, infinities in the
gradient and in the keys and values that the others see among them."""
import math

import pytest
import torch

from test_gpu_train import Problem, bytes_, dlo, float32_by_default, stream  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")

CASES = [
    # B, H, G, hd, nq, nk, causal block, q_lens, k_lens
    (2, 4, 2, 64, 300, 300, 0, [170, 300], [300, 190]),
    (2, 2, 2, 128, 300, 260, 50, [170, 290], [200, 190]),
    (2, 16, 16, 72, 700, 300, 0, [500, 1], [1, 300]),       # two CTAs per SM
    (2, 2, 1, 40, 300, 100, 0, [170, 300], [100, 60]),      # one key tile
    (1, 2, 2, 64, 400, 150, 1, None, None),                 # the first 250 queries see nothing
    (2, 16, 4, 64, 40, 1500, 0, [30, 40], [1500, 1100]),    # the keys split, heads share query tiles
    (1, 2, 2, 96, 2500, 100, 0, [2400], [70]),              # dK and dV split over the queries
    (1, 1, 1, 80, 200, 300, 1, [90], None),                 # the last keys are seen by nobody
]


def unused_rows(p):
    """Truth values [B, nq] and [B, nk]: queries that see nothing, keys that nothing sees."""
    B, H, G, hd, nq, nk, cb = p.c
    i, j = torch.arange(nq, device="cuda")[:, None] + nk - nq, torch.arange(nk, device="cuda")[None]
    q, k = [], []
    for b in range(B):
        see = (torch.arange(nq, device="cuda")[:, None] < p.ql[b]) & (j < p.kl[b])
        if cb:
            see = see & (i >= 0) & (torch.div(i, cb, rounding_mode="floor") >= torch.div(j, cb, rounding_mode="floor"))
        q.append(~see.any(1))
        k.append(~see.any(0))
    return torch.stack(q), torch.stack(k)


def infinities(case):
    p = Problem(*case, seed=31, fused=False)
    q_out, k_out = unused_rows(p)
    assert q_out.any() or k_out.any()
    for b in range(p.c[0]):
        # the last key and value that somebody sees, the last query that sees something: in the tile where the others end
        j = int((~k_out[b]).nonzero()[-1])
        i = int((~q_out[b]).nonzero()[-1])
        p.k[b, j], p.v[b, j], p.q[b, i], p.do[b, i] = INF, -INF, INF, INF
    return p, q_out, k_out


IDS = ["x".join(map(str, c[:7])) + ("-lens" if c[7] or c[8] else "") for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_rows_that_see_nothing_are_zero_beside_infinities(case):
    p, q_out, _ = infinities(case)
    p.forward()
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    assert (p.o[q_out] == 0).all(), "O"
    assert (p.lse.transpose(1, 2)[q_out] == -math.inf).all(), "lse"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradients_of_rows_without_a_part_are_zero_beside_infinities(case):
    p, q_out, k_out = infinities(case)
    p.forward()
    grads = p.grads()
    p.backward(grads)
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    assert (grads[0][q_out] == 0).all(), "dQ"
    assert (grads[1][k_out] == 0).all(), "dK"
    assert (grads[2][k_out] == 0).all(), "dV"
