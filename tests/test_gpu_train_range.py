"""Attention training ops where the numbers get large: row maxima that jump
from tile to tile, logits and products with a large common part, and
tensor-wide error bounds beside the element-wise ones.

u = 2^-8 is half a bf16 step relative to the value.  A score is a sum of at most
nine tensor-core steps (head dim / 16 and the row statistic), each off by at most 2^-22 of
the magnitudes that it adds (17 terms, cut to 24 bits of the largest), and is
compared with an lse of the same kind: exp(s - L) is off, relatively, by at
most 2 * 9 * 2^-22 (A + |L|) <= f = 2^-17.8 (A + |L|) + 2^-20, where A = sum_d |q k| / sqrt(hd)
and 2^-20 stands for the exponential and its argument's product.

A rounding to bf16 is off by at most u and, over many values, by u / sqrt(3) in
the root mean square; independent ones add in squares.  So the relative 2-norm
error of a tensor behind r roundings is at most u sqrt(r / 3): O and dV have two
(P, the result), dQ and dK three (D through O, dS, the result).
"""
import math

import pytest
import torch

from test_gpu_train import NAN, U, Problem, bytes_, dlo, float32_by_default, stream, within  # noqa: F401

pytestmark = pytest.mark.gpu

G = 2.0 ** -17.8
u = 2.0 ** -8


def heads_of(p, b):
    """(query head, key/value head, visible pairs, q, k, v, do) of sequence b in 64 bits, what lies behind the lengths zero."""
    B, H, Gr, hd, nq, nk, cb = p.c
    i, j = torch.arange(nq, device="cuda")[:, None] + nk - nq, torch.arange(nk, device="cuda")[None]
    see = (torch.arange(nq, device="cuda")[:, None] < p.ql[b]) & (j < p.kl[b])
    if cb:
        see = see & (i >= 0) & (torch.div(i, cb, rounding_mode="floor") >= torch.div(j, cb, rounding_mode="floor"))

    def part(t, n, w):
        return torch.where(torch.arange(t.shape[1], device="cuda")[:, None] < n[b], t[b, :, w * hd:(w + 1) * hd].double(), 0.0)

    for h in range(H):
        g = h // (H // Gr)
        yield h, g, see, part(p.q, p.ql, h), part(p.k, p.kl, g), part(p.v, p.kl, g), part(p.do, p.ql, h)


def exact(p):
    """O, lse, dQ, dK, dV in 64 bits and their element-wise bounds (see above; D from the O that the forward left)."""
    B, H, Gr, hd, nq, nk, _ = p.c
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")                    # noqa: E731
    r = {k: z(B, nq, H, hd) for k in ("o", "dq", "o_b", "dq_b")} | {k: z(B, nk, Gr, hd) for k in ("dk", "dv", "dk_b", "dv_b")}
    r["lse"] = torch.full((B, H, nq), -math.inf, dtype=torch.float64, device="cuda")
    r["lse_b"] = z(B, H, nq)
    for b in range(B):
        for h, g, see, q, k, v, do in heads_of(p, b):
            s = (q @ k.T / math.sqrt(hd)).masked_fill(~see, -math.inf)
            any_ = see.any(1)
            lse = torch.where(any_, torch.logsumexp(s, 1), -math.inf)
            mid = torch.where(any_, lse, 0.0)[:, None]
            pr = torch.where(see, torch.exp(s - mid), 0.0)
            f = torch.where(see, G * (q.abs() @ k.abs().T / math.sqrt(hd) + mid.abs()) + 2.0 ** -20, 0.0)
            o = pr @ v
            top = f.amax(1, keepdim=True)                       # of the sum that divides
            o_b = ((U + f + top) * pr) @ v.abs() + U * o.abs() + 1e-30
            r["lse"][b, h], r["lse_b"][b, h], r["o"][b, :, h], r["o_b"][b, :, h] = lse, top[:, 0], o, o_b
            r["dv"][b, :, g] += pr.T @ do
            r["dv_b"][b, :, g] += ((U + f) * pr).T @ do.abs()
            D = (do * o).sum(1, keepdim=True)
            ds = pr * (do @ v.T - D)
            e = (do.abs() * o_b).sum(1, keepdim=True) + 2.0 ** -17.8 * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True))
            ds_b = (U + f) * ds.abs() + pr * e
            r["dq"][b, :, h] = ds @ k / math.sqrt(hd)
            r["dq_b"][b, :, h] = ds_b @ k.abs() / math.sqrt(hd) + U * r["dq"][b, :, h].abs() + 1e-30
            r["dk"][b, :, g] += ds.T @ q / math.sqrt(hd)
            r["dk_b"][b, :, g] += ds_b.T @ q.abs() / math.sqrt(hd)
    for x in ("dk", "dv"):
        r[x + "_b"] += U * r[x].abs() + 1e-30
    return r


def both_passes(p):
    p.forward()
    grads = p.grads()
    p.backward(grads)
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    return grads


def check(p, grads, r):
    for name, got in (("o", p.o), ("dq", grads[0]), ("dk", grads[1]), ("dv", grads[2])):
        within(got.reshape(r[name].shape), r[name], r[name + "_b"], name)
    empty = r["lse"] == -math.inf
    assert torch.equal(p.lse == -math.inf, empty)
    assert ((p.lse.double() - r["lse"]).abs()[~empty] <= r["lse_b"][~empty]).all(), "lse"


def off(got, want):
    return float((got.double().reshape(want.shape) - want).norm() / want.norm())


# ------------------------------------------------------------------ maxima that jump

JUMPS = [
    (1, 4, 4, 128, 300, 896, 0, None, None),              # one CTA a tile
    (1, 2, 2, 64, 260, 1100, 0, None, None),              # the keys of a tile split
    (2, 16, 16, 72, 700, 1100, 0, None, None),            # two CTAs per SM
    (2, 16, 16, 64, 700, 1100, 1, None, None),            # likewise, token-causal
    (2, 4, 2, 128, 600, 600, 100, [600, 400], [600, 500]),
    (2, 16, 2, 64, 20, 1100, 0, [20, 11], [1100, 777]),   # heads of a group share query tiles, keys split
    (1, 8, 2, 80, 50, 700, 1, None, None),                # likewise, causal, not split
    (1, 2, 2, 96, 700, 500, 1, None, None),               # the first 200 queries see nothing
]


@pytest.mark.parametrize("case", JUMPS, ids=lambda c: "x".join(map(str, c[:7])) + ("-lens" if c[7] else ""))
def test_row_maxima_that_jump_from_tile_to_tile(case):
    """In every tile of 128 keys one key answers to its own column of q with logits of
    deviation 6, among others of deviation 1: about one row in twelve jumps by more than
    2^8 at a tile, several times on its way, while what it had keeps its weight."""
    p = Problem(*case, seed=11, fused=False)
    B, H, Gr, hd, nq, nk, cb = p.c
    tiles = (nk + 127) // 128
    assert tiles <= hd
    for t in range(tiles):
        j = min(128 * t + 37, nk - 1)
        for g in range(Gr):
            spike = torch.zeros(hd, device="cuda")
            spike[t] = 6.0 * math.sqrt(hd)
            for b in range(B):
                if j < p.kl[b]:
                    p.k[b, j, g * hd:(g + 1) * hd] = spike.to(torch.bfloat16)
    r = exact(p)
    # the inputs do what they are for: some rows rise by more than 8 (in units of log 2) after their first tile, twice where there are many
    jumps = 0
    for h, g, see, q, k, v, do in heads_of(p, 0):
        s = (q @ k.T / math.sqrt(hd) / math.log(2)).masked_fill(~see, -math.inf)
        m = torch.stack([x.amax(1) for x in s.split(128, 1)], 1)
        m = m[torch.isfinite(m[:, 0])]
        top = torch.cummax(m, 1).values
        jumps = max(jumps, int((m[:, 1:] > top[:, :-1] + 8).sum(1).max()))
    assert jumps >= (2 if tiles > 6 else 1)
    check(p, both_passes(p), r)


# ------------------------------------------------------------------ large common parts

def _last_two(p, b, t, first, second, heads):
    """The last two columns of every head of rows [0, n) of t (both lie in the last step of a product)."""
    hd = p.c[3]
    for h in range(heads):
        t[b, :, (h + 1) * hd - 2] = first
        t[b, :, (h + 1) * hd - 1] = second


def _gradients(q, k, v, do, hd, lse_to=lambda x: x, d_to=lambda x: x):
    s = q @ k.T / math.sqrt(hd)
    lse = torch.logsumexp(s, 1, keepdim=True)
    pr = torch.exp(s - lse_to(lse * math.sqrt(hd)) / math.sqrt(hd))
    D = (do * (torch.softmax(s, 1) @ v)).sum(1, keepdim=True)
    ds = pr * (do @ v.T - d_to(D))
    return ds @ k / math.sqrt(hd), ds.T @ q / math.sqrt(hd), pr.T @ do


def two_parts(x):
    """x as the sum of two bf16 values: what is left of three without the last."""
    a = x.to(torch.bfloat16).double()
    return a + (x - a).to(torch.bfloat16).double()


@pytest.mark.parametrize("hd", [64, 72, 128])
@pytest.mark.parametrize("what", ["logits", "products"])
def test_row_statistics_of_the_backward_pass_hold_24_bits(what, hd):
    """Logits of 6000 to 16000 (dO V^T of 33000 to 66000), nearly all of it common to a row's keys.
    It comes in with a product's last step and goes with the row statistic, one step later, so what
    fp32 adds is a few of its units: of a magnitude x at most 4 * 2^-23 x for P (the step, the
    statistic's, lse and its form in raw units) and 8 * 2^-23 x for dP - D (the step, the statistic's,
    the sum P dP of D with P off by 2^-22).  With the last of the statistic's three parts left out the
    oracle misses the bound of dK."""
    H, nq, nk = 2, 300, 128
    p = Problem(1, H, H, hd, nq, nk, seed=5, fused=False)
    g = torch.Generator(device="cuda").manual_seed(hd)
    if what == "logits":
        # multiples of 512, which bf16 holds, and 192, which needs the second part and leaves work for the third
        _last_two(p, 0, p.q, (256 + 2 * torch.randint(0, 128, (nq,), generator=g, device="cuda")).to(torch.bfloat16), 16.0, H)
        _last_two(p, 0, p.k, 256.0, 12.0, H)
        _last_two(p, 0, p.v, 0.0, 0.0, H)
    else:
        p.do.mul_(5.0)                                   # of deviation 1/2
        _last_two(p, 0, p.do, (32 + torch.randint(0, 128, (nq,), generator=g, device="cuda") / 4).to(torch.bfloat16), 10.0, H)
        _last_two(p, 0, p.v, 1024.0, 10.0, H)
    got = both_passes(p)
    for h, _, _, q, k, v, do in heads_of(p, 0):
        at = slice(h * hd, (h + 1) * hd - 2)             # the last two columns carry the common part
        want = _gradients(q, k, v, do, hd)
        poor = _gradients(q, k, v, do, hd, **({"lse_to": two_parts} if what == "logits" else {"d_to": two_parts}))
        s = q @ k.T / math.sqrt(hd)
        pr, dp = torch.softmax(s, 1), do @ v.T
        D = (pr * dp).sum(1, keepdim=True)
        size = float(s.abs().max()) if what == "logits" else float((pr * D).norm() / (pr * (dp - D)).norm())
        more = (4 if what == "logits" else 8) * 2.0 ** -23 * size
        for name, x, y, z, r in zip(("dq", "dk", "dv"), got, want, poor, (3, 3, 2)):
            y, z = y[:, :hd - 2], z[:, :hd - 2]
            if name == "dv" and what == "products":
                more = 0.0
            bound = u * math.sqrt(r / 3) + more
            assert off(x[0, :, at], y) <= bound, name
            if name == "dk":
                assert off(z, y) > bound, "the bound would not show a lost part"


# ------------------------------------------------------------------ over whole tensors

@pytest.mark.parametrize("case", [(2, 16, 16, 72, 1024, 1024, 0, None, None), (1, 4, 4, 128, 1100, 1100, 1, None, None),
                                  (2, 8, 2, 64, 300, 1500, 0, None, None), (2, 16, 4, 64, 40, 1500, 0, None, None),
                                  (1, 6, 3, 96, 900, 200, 0, None, None), (2, 4, 2, 80, 520, 520, 104, [520, 312], [520, 301])],
                         ids=lambda c: "x".join(map(str, c[:7])) + ("-lens" if c[7] else ""))
def test_errors_over_whole_tensors_are_those_of_the_roundings(case):
    p = Problem(*case, seed=21)
    got = both_passes(p)
    r = exact(p)
    for name, x, n in (("o", p.o, 2), ("dq", got[0], 3), ("dk", got[1], 3), ("dv", got[2], 2)):
        assert off(x, r[name]) <= u * math.sqrt(n / 3), name


# ------------------------------------------------------------------ lengths that change under a graph

@pytest.mark.parametrize("case", [(2, 16, 4, 64, 40, 1500, 0), (2, 4, 2, 64, 300, 300, 50), (2, 16, 16, 72, 700, 700, 0)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_forward_and_backward_follow_inputs_and_lengths_that_change_in_place(case, graph):
    """Inputs, lengths among them, are overwritten right before each pair of calls; the first shape's forward splits its keys."""
    nq, nk = case[4:6]
    lens = [([nq, nq - 19], [nk - 5, nk]), ([nq - 33, nq], [nk, nk - 140]), ([nq - 1, 1], [1, nk - 1]), ([0, nq], [nk, 0])]
    sets = [Problem(*case, *lens[i], seed=60 + i, fused=False) for i in range(4)]
    want = [(s.o, s.lse, *both_passes(s)) for s in sets]
    p = Problem(*case, *lens[0], seed=60, fused=False)
    grads = p.grads()
    wf, wb = p.forward(), p.backward(grads)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")

    def one_round():
        for s, w in zip(sets, want):
            for n in ("q", "k", "v", "do", "q_lens", "k_lens"):
                getattr(p, n).copy_(getattr(s, n))
            p.forward(wf)
            p.backward(grads, wb)
            for x, y in zip((p.o, p.lse, *grads), w):
                differ.add_((x != y).sum())

    one_round()
    torch.cuda.synchronize()
    assert int(differ.item()) == 0
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one_round()
        one_round = g.replay
    for _ in range(10):
        one_round()
    assert int(differ.item()) == 0 and int(p.err.item()) == 0
