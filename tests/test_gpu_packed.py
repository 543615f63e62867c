"""Operators for packed batches against plain forms in 64 bits.

Attention bounds are element-wise and follow from the roundings: u = 2^-8 is half a
bf16 step relative to the value.  With P, dS rounded to bf16 before their products
and O as the forward left it:
  |O err|  <= u (sum_j p |v| + |o|) =: o_b
  |dV err| <= u (sum_i p |do| + |dv|)
  |D err|  <= sum_d |do| o_b =: e,   |dS err| <= u |dS| + p e
  |dQ err| <= (sum_j (u |dS| + p e) |k|) / sqrt(hd) + u |dQ|, and dK likewise
plus what fp32 adds: a score off by ~2^-22 (sum_d |q k|) / sqrt(hd) is f = 2^-18
relative in p where |q|.|k| / sqrt(hd) <= 16, and dP is off by 2^-20 sum_d |do v|.
u is taken 1% larger for products of two roundings.

Rotary positions: the result's rounding, u; angles are exact to 2^-32 of a turn, sine
and cosine and the two products to 2^-20 of (|u| + |v|) amp together.
"""
import math

import numpy as np
import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

pytestmark = pytest.mark.gpu

U = 1.01 * 2.0 ** -8
F = 2.0 ** -18
NAN = float("nan")
DEV = "cuda"
KEEP = 3.5             # what output buffers hold before a call


@pytest.fixture(autouse=True)
def float32_by_default():
    """Another test module of the same process may have set another default."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def stream():
    return torch.cuda.current_stream().cuda_stream


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts_of(lens, lead=0):
    return [lead] + (lead + np.cumsum(lens)).tolist() if len(lens) else [lead]


def scratch(n):
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)     # NaN where read unwritten


def within(y, ref, bound, name):
    d = (y.double() - ref).abs()
    assert torch.isfinite(d).all(), f"{name}: not finite"
    over = float((d / bound).max()) if d.numel() else 0.0
    assert over <= 1, f"{name}: error {over:.3f} of its bound"


class Packed:
    """Packed sequences in buffers with rows before and behind them, and a 64-bit reference."""

    def __init__(self, H, G, hd, ql, kl=None, cb=0, lead=0, slack=0, pad=0, seed=0, scale=1.0):
        self.c = (H, G, hd, cb)
        g = torch.Generator(device=DEV).manual_seed(seed + 7 * sum(ql) + hd)
        self.ql, self.kl = list(ql), list(ql if kl is None else kl)
        self.qs, self.ks = starts_of(self.ql, lead), starts_of(self.kl, lead)
        self.rq, self.rk = self.qs[-1] + slack, self.ks[-1] + slack
        self.rq, self.rk = max(self.rq, 1), max(self.rk, 1)
        self.q_starts = int32(self.qs)
        self.k_starts = self.q_starts if kl is None else int32(self.ks)

        def rnd(rows, cols, s=1.0):
            return (torch.randn((rows, cols), generator=g, device=DEV) * s).to(torch.bfloat16)

        if kl is None:
            rows = rnd(self.rq, (H + 2 * G) * hd + pad, scale)
            self.q, self.k, self.v = rows[:, :H * hd], rows[:, H * hd:(H + G) * hd], rows[:, (H + G) * hd:(H + 2 * G) * hd]
        else:
            self.q = rnd(self.rq, H * hd + pad, scale)[:, :H * hd]
            kv = rnd(self.rk, 2 * G * hd + pad, scale)
            self.k, self.v = kv[:, :G * hd], kv[:, G * hd:2 * G * hd]
        self.do = rnd(self.rq, H * hd + pad, 0.1)[:, :H * hd]
        for t, s in ((self.q, self.qs), (self.do, self.qs), (self.k, self.ks), (self.v, self.ks)):
            t[:s[0]] = NAN                          # rows of no sequence are never used
            t[s[-1]:] = NAN
        self.o = torch.full((self.rq, H * hd + pad), KEEP, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((H, self.rq), KEEP, device=DEV)
        self.g = [torch.full((r, w * hd + pad), KEEP, dtype=torch.bfloat16, device=DEV)
                  for r, w in ((self.rq, H), (self.rk, G), (self.rk, G))]
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def desc(self):
        H, G, hd, cb = self.c
        return dlo.make_attn_packed(batch=self.q_starts.numel() - 1, heads=H, kv_heads=G, head_dim=hd, rows_q=self.rq, rows_k=self.rk,
                                    causal_block=cb, ldq=self.q.stride(0), ldk=self.k.stride(0), ldv=self.v.stride(0),
                                    ldo=self.o.stride(0), lddq=self.g[0].stride(0), lddk=self.g[1].stride(0),
                                    lddv=self.g[2].stride(0), lddo=self.do.stride(0), q_starts=self.q_starts.data_ptr(),
                                    k_starts=self.k_starts.data_ptr())

    def forward(self, ws=None):
        a = self.desc()
        ws = scratch(dlo.dlo_attention_packed_fwd_workspace_bytes(a)) if ws is None else ws
        dlo.dlo_op_attention_packed_fwd(a, self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.o.data_ptr(),
                                        self.lse.data_ptr(), ws.data_ptr(), ws.numel(), self.err.data_ptr(), stream())
        return ws

    def backward(self, ws=None):
        a = self.desc()
        ws = scratch(dlo.dlo_attention_packed_bwd_workspace_bytes(a)) if ws is None else ws
        dlo.dlo_op_attention_packed_bwd(a, self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.o.data_ptr(),
                                        self.lse.data_ptr(), self.do.data_ptr(), *(t.data_ptr() for t in self.g),
                                        ws.data_ptr(), ws.numel(), self.err.data_ptr(), stream())
        return ws

    def reference(self):
        """O, lse, dQ, dK, dV in 64 bits and their error bounds."""
        H, G, hd, cb = self.c
        z = lambda r, w: torch.zeros((r, w, hd), dtype=torch.float64, device=DEV)      # noqa: E731
        out = {k: z(self.rq, H) for k in ("o", "dq", "o_b", "dq_b")}
        out |= {k: z(self.rk, G) for k in ("dk", "dv", "dk_b", "dv_b")}
        out["lse"] = torch.full((H, self.rq), -math.inf, dtype=torch.float64, device=DEV)
        heads = lambda t, n, s, h: t[s:s + n, h * hd:(h + 1) * hd].double()          # noqa: E731
        for nq, nk, q0, k0 in zip(self.ql, self.kl, self.qs, self.ks):
            i = torch.arange(nq, device=DEV)[:, None] + nk - nq
            j = torch.arange(nk, device=DEV)[None]
            see = torch.ones((nq, nk), dtype=torch.bool, device=DEV)
            if cb:
                see = (i >= 0) & (torch.div(i, cb, rounding_mode="floor") >= torch.div(j, cb, rounding_mode="floor"))
            any_ = see.any(1) if nk else torch.zeros(nq, dtype=torch.bool, device=DEV)
            rq, rk = slice(q0, q0 + nq), slice(k0, k0 + nk)
            for h in range(H):
                g = h // (H // G)
                q, do = heads(self.q, nq, q0, h), heads(self.do, nq, q0, h)
                k, v = heads(self.k, nk, k0, g), heads(self.v, nk, k0, g)
                s = (q @ k.T / math.sqrt(hd)).masked_fill(~see, -math.inf)
                lse = torch.where(any_, torch.logsumexp(s, 1) if nk else torch.zeros(nq, dtype=torch.float64, device=DEV), -math.inf)
                p = torch.where(see, torch.exp(s - torch.where(any_, lse, 0.0)[:, None]), 0.0)
                o = p @ v
                out["lse"][h, rq] = lse
                out["o"][rq, h] = o
                o_b = (U + F) * (p @ v.abs()) + U * o.abs() + 1e-30
                out["o_b"][rq, h] = o_b
                out["dv"][rk, g] += p.T @ do
                out["dv_b"][rk, g] += (U + F) * (p.T @ do.abs())
                dp = do @ v.T
                D = (do * o).sum(1, keepdim=True)
                e = (do.abs() * o_b).sum(1, keepdim=True)
                ds = p * (dp - D)
                ds_b = (U + F) * ds.abs() + p * (e + 2.0 ** -20 * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True)))
                out["dq"][rq, h] = ds @ k / math.sqrt(hd)
                out["dq_b"][rq, h] = ds_b @ k.abs() / math.sqrt(hd) + U * out["dq"][rq, h].abs() + 1e-30
                out["dk"][rk, g] += ds.T @ q / math.sqrt(hd)
                out["dk_b"][rk, g] += ds_b.T @ q.abs() / math.sqrt(hd)
        for x in ("dk", "dv"):
            out[x + "_b"] += U * out[x].abs() + 1e-30
        return out

    def check(self, ref, grads=False):
        H, G, hd, _ = self.c
        assert int(self.err.item()) == 0
        rows = {"q": slice(self.qs[0], self.qs[-1]), "k": slice(self.ks[0], self.ks[-1])}
        todo = [(self.o, "o", H, "q")]
        if grads:
            todo += [(self.g[0], "dq", H, "q"), (self.g[1], "dk", G, "k"), (self.g[2], "dv", G, "k")]
        for y, name, w, of in todo:
            r = rows[of]
            within(y[r, :w * hd].unflatten(1, (w, hd)), ref[name][r], ref[name + "_b"][r], name)
            assert bool((y[:r.start] == KEEP).all() and (y[r.stop:] == KEEP).all() and (y[:, w * hd:] == KEEP).all()), f"{name}: others' rows"
        r = rows["q"]
        assert bool((self.lse[:, :r.start] == KEEP).all() and (self.lse[:, r.stop:] == KEEP).all()), "lse: others' rows"
        lse, want = self.lse[:, r], ref["lse"][:, r]
        empty = want == -math.inf
        assert torch.equal(lse == -math.inf, empty), "empty rows"
        d = (lse.double() - want)[~empty]
        # scores of magnitude <= 16 in fp32 products, exp and log within a few ulp
        assert d.numel() == 0 or float(d.abs().max()) <= 1e-5


CASES = [
    # H, G, hd, q lengths, k lengths, causal block, rows before, behind
    (1, 1, 8, [1], None, 0, 0, 0),
    (2, 2, 64, [128, 128], None, 0, 0, 0),
    (2, 2, 64, [127, 1, 129, 0, 300], None, 0, 0, 0),
    (2, 1, 128, [5, 250, 131], None, 0, 3, 7),
    (4, 4, 72, [257, 64, 33], None, 0, 130, 1),
    (3, 3, 80, [200], [385], 0, 0, 5),
    (2, 2, 128, [100, 300, 0, 20], [256, 129, 50, 0], 0, 1, 1),
    (2, 2, 16, [260, 3, 130], None, 1, 0, 0),
    (4, 1, 64, [300, 171], None, 1, 9, 9),
    (2, 2, 96, [150, 10], [400, 1], 1, 0, 0),                  # the first nine queries of the second see nothing
    (2, 2, 112, [400], [150], 1, 0, 0),
    (2, 2, 128, [600, 520, 77], None, 100, 0, 0),
    (2, 2, 72, [513, 300], [500, 301], 170, 0, 2),
    (2, 2, 88, [260, 130], None, 1 << 30, 0, 0),               # one block: every key
    (6, 2, 64, [1] * 40, [37] * 39 + [900], 0, 0, 0),          # single queries, more sequences than lanes
    (40, 8, 128, [1, 1, 1, 1], [300, 1, 0, 700], 1, 0, 0),     # groups of five share a tile
    (10, 2, 64, [300, 3, 26], None, 1, 0, 3),
    (24, 2, 64, [10, 11], [700, 90], 1, 0, 0),                 # groups of twelve
    (3, 1, 40, [43, 44, 1], None, 0, 0, 0),                    # 42 queries a tile, two rows empty
    (2, 1, 64, [5], [4100], 0, 0, 0),                          # few queries: the keys are split
    (2, 2, 128, [17, 0, 9], [5000, 10, 300], 1, 2, 2),
    (2, 2, 64, [2500], [100], 0, 0, 0),                        # few keys: their gradients are split
    (2, 2, 64, [1500, 900], [70, 0], 0, 4, 4),
    (4, 2, 72, [1500, 900], None, 1, 0, 0),                    # causal: likewise
    (8, 2, 128, [33, 7], [1300, 515], 0, 0, 0),
    (1, 1, 64, [3] * 300, None, 0, 0, 0),
    (16, 4, 64, [1000, 1], None, 1, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%dx%d-%d-%s-%d" % (c[0], c[1], c[2], sum(c[3]), c[4] and sum(c[4]), c[5]))
def test_attention(case):
    H, G, hd, ql, kl, cb, lead, slack = case
    p = Packed(H, G, hd, ql, kl, cb, lead, slack, pad=8 if lead else 0)
    ref = p.reference()
    p.forward()
    p.check(ref)
    p.backward()
    p.check(ref, grads=True)


@pytest.mark.parametrize("hd", [8, 24, 48, 64, 72, 104, 120, 128])
def test_head_dims(hd):
    p = Packed(2, 1, hd, [140, 0, 61], None, 1, 1, 1)
    ref = p.reference()
    p.forward()
    p.backward()
    p.check(ref, grads=True)


def test_two_calls_give_the_same_bits():
    a, b = (Packed(8, 2, 64, [700, 31, 0, 400], None, 1) for _ in range(2))
    for p in (a, b):
        p.forward()
        p.backward()
    for x, y in zip([a.o, a.lse] + a.g, [b.o, b.lse] + b.g):
        assert torch.equal(x, y)


@pytest.mark.parametrize("value", [math.inf, -math.inf, NAN])
@pytest.mark.parametrize("cb", [0, 1])
def test_a_sequence_keeps_to_itself(value, cb):
    """Infinities and NaN in one sequence reach no other one, to the bit."""
    clean, dirty = (Packed(4, 2, 72, [130, 77, 200], None, cb) for _ in range(2))
    for t in (dirty.q, dirty.k, dirty.v, dirty.do):
        t[130:207] = value
    for p in (clean, dirty):
        p.forward()
        p.backward()
    for x, y in zip([clean.o] + clean.g, [dirty.o] + dirty.g):
        assert torch.equal(x[:130], y[:130]) and torch.equal(x[207:], y[207:])
    assert torch.equal(clean.lse[:, :130], dirty.lse[:, :130]) and torch.equal(clean.lse[:, 207:], dirty.lse[:, 207:])


@pytest.mark.parametrize("kl", [[300], [5000], [40]])
def test_one_sequence_is_the_padded_op(kl):
    """The same tiles in the same order where no heads share one: the same bits."""
    H, hd, nq, nk = 2, 64, 170, kl[0]
    p = Packed(H, H, hd, [nq], kl, 1)
    p.forward()
    p.backward()
    o, lse = torch.empty_like(p.o), torch.empty_like(p.lse)
    g = [torch.empty_like(t) for t in p.g]
    a = dlo.make_attn(batch=1, heads=H, head_dim=hd, nq=nq, nk=nk, causal_block=1, ldq=p.q.stride(0), ldk=p.k.stride(0),
                      ldv=p.v.stride(0), ldo=o.stride(0), lddq=g[0].stride(0), lddk=g[1].stride(0), lddv=g[2].stride(0),
                      lddo=p.do.stride(0))
    ws = scratch(max(dlo.dlo_attention_fwd_workspace_bytes(a), dlo.dlo_attention_bwd_workspace_bytes(a)))
    dlo.dlo_op_attention_fwd(a, p.q.data_ptr(), p.k.data_ptr(), p.v.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                             ws.numel(), p.err.data_ptr(), stream())
    ref = p.reference()
    p.check(ref, grads=True)
    within(o.unflatten(1, (H, hd)), ref["o"], ref["o_b"], "padded O")


def test_starts_out_of_range_touch_nothing_outside():
    """Starts are taken into 0 .. rows: here the last sequence ends with the buffer."""
    p = Packed(2, 2, 64, [100, 60], None, 0)
    p.q_starts.copy_(int32([-5, 100, 1 << 30]))
    ref = p.reference()
    p.forward()
    p.backward()
    p.check(ref, grads=True)


def test_attention_gradients_against_differences():
    """The directional derivative that the gradients give against a quotient of the 64-bit loss.  Each gradient
    element is off by its bound at most, so the derivative by sum bound |direction|; the quotient itself by
    the third derivative times step^2, below 1e-6 of the loss's scale here."""
    p = Packed(2, 1, 32, [40, 21], [50, 33], 1, scale=0.5)
    ref = p.reference()
    p.forward()
    p.backward()
    H, G, hd, _ = p.c
    gen = torch.Generator(device=DEV).manual_seed(5)
    for t, name, w, g in ((p.q, "dq", H, p.g[0]), (p.k, "dk", G, p.g[1]), (p.v, "dv", G, p.g[2])):
        d = torch.randn(t.shape, generator=gen, device=DEV, dtype=torch.float64)
        losses = []
        exact, attr = t.double(), name[1]
        for e in (1e-4, -1e-4):
            setattr(p, attr, exact + e * d)
            losses.append(float((p.reference()["o"].flatten(1) * p.do.double()).sum()))
        setattr(p, attr, t)
        slope = (losses[0] - losses[1]) / 2e-4
        got = float((g.double() * d).sum())
        limit = float((ref[name + "_b"].flatten(1) * d.abs()).sum()) + 1e-6 * float(p.do.double().abs().sum())
        assert abs(got - slope) <= limit, name


# ------------------------------------------------------------------ plan

def plan(grids, offsets, rows, room=None):
    axes = len(grids[0])
    g = int32(grids)
    o = None if offsets is None else int32(offsets)
    starts = torch.full((len(grids) + 1,), -7, dtype=torch.int32, device=DEV)
    positions = torch.full((room or rows, axes), -7, dtype=torch.int32, device=DEV)
    dlo.dlo_op_packed_plan(g.data_ptr(), None if o is None else o.data_ptr(), len(grids), axes, rows, starts.data_ptr(),
                           positions.data_ptr(), stream())
    return starts.tolist(), positions.cpu().numpy()


def plan_reference(grids, offsets, rows, room=None):
    axes = len(grids[0])
    starts, positions, n = [0], np.full((room or rows, axes), -7, dtype=np.int64), 0
    for b, grid in enumerate(grids):
        total = math.prod(max(0, e) for e in grid)
        for i in range(min(total, rows - n)):
            place = np.unravel_index(i, grid)
            positions[n] = [int(x) + (offsets[b][a] if offsets else 0) for a, x in enumerate(place)]
            n += 1
        starts.append(n)
    return starts, positions


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("batch", [1, 7, 255, 256, 257, 700])
def test_plan(axes, batch):
    rng = np.random.default_rng(axes * 1000 + batch)
    grids = rng.integers(-1, 7 if axes < 3 else 4, (batch, axes)).tolist()
    grids[0] = [60, 3, 2, 4][:axes]
    offsets = rng.integers(-9, 1 << 20, (batch, axes)).tolist()
    total = plan_reference(grids, None, 1 << 30, 1 << 16)[0][-1]
    for at, rows in ((offsets, total + 9), (None, total), (offsets, max(1, total - 11)), (offsets, 5)):
        want, got = plan_reference(grids, at, rows, total + 20), plan(grids, at, rows, total + 20)
        assert got[0] == want[0]
        assert np.array_equal(got[1], want[1])


def test_plan_of_long_sequences_and_large_extents():
    starts, positions = plan([[100000], [1 << 30], [5]], [[3], [-7], [0]], 250000)
    assert starts == [0, 100000, 250000, 250000]
    assert np.array_equal(positions[:, 0], np.concatenate([np.arange(100000) + 3, np.arange(150000) - 7]))
    starts, positions = plan([[1 << 30, 1 << 30, 1 << 30, 1 << 30]], None, 100)
    assert starts == [0, 100] and np.array_equal(positions[:, 3], np.arange(100)) and not positions[:, :3].any()
    starts, _ = plan([[2, 3]] * 65535, None, 1 << 19)
    assert starts == [min(6 * i, 1 << 19) for i in range(65536)]


def test_plan_without_positions():
    g, starts = int32([[4, 5]] * 300), torch.zeros(301, dtype=torch.int32, device=DEV)
    dlo.dlo_op_packed_plan(g.data_ptr(), None, 300, 2, 100000, starts.data_ptr(), None, stream())
    assert starts.tolist() == [20 * i for i in range(301)]


# ------------------------------------------------------------------ rotary positions

def angles(r, positions):
    """Radians of every pair of every row: whole turns taken off in Python's integers (a 64-bit float would lose
    2^-20 at position 2^31).  The table of steps against its formulas is another test."""
    steps = dlo.dlo_rope_steps(r).view(np.uint64).tolist()
    axis = axis_of(r)
    turns = [[(n[a] * s % (1 << 64)) / 2.0 ** 64 for a, s in zip(axis, steps)] for n in positions.tolist()]
    return torch.tensor(turns, dtype=torch.float64, device=DEV) * (2 * math.pi)


def axis_of(r):
    return [a for a in range(r.axes) for _ in range(r.axis[a].dim // 2)]


def rope_reference(r, x, positions, back=False):
    """x [rows, heads * hd] in 64 bits and the size of what was added up."""
    H, hd, n = r.heads, r.head_dim, len(axis_of(r))
    angle = angles(r, positions) * (-1 if back else 1)
    c, s = r.amp * angle.cos()[:, None], r.amp * angle.sin()[:, None]
    x = x.double().unflatten(1, (H, hd))
    y, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(n, device=DEV)
    u, v = (2 * i, 2 * i + 1) if r.layout == dlo.ROPE_INTERLEAVED else (i, i + n)
    a, b = x[..., u], x[..., v]
    y[..., u], y[..., v] = a * c - b * s, a * s + b * c
    size[..., u] = size[..., v] = (a.abs() + b.abs()) * abs(r.amp)
    return y.flatten(1), size.flatten(1)


ROPES = [
    # heads, head_dim, dims, rows
    (1, 8, [2], 1), (1, 8, [8], 5), (3, 64, [64], 33), (2, 128, [44, 42, 42], 70), (5, 72, [72], 130), (5, 72, [24, 24, 24], 9),
    (2, 96, [20], 50), (7, 40, [2, 6], 20), (4, 80, [40], 300), (40, 128, [128], 3), (1, 256, [254], 4), (1, 256, [2], 7),
    (2, 128, [60, 60], 31), (3, 32, [10, 8, 2, 8], 65), (80, 128, [128], 1), (300, 64, [32], 2), (6, 24, [12], 1000),
    (2, 48, [28], 17),
]


@pytest.mark.parametrize("layout", [dlo.ROPE_INTERLEAVED, dlo.ROPE_HALF], ids=["interleaved", "half"])
@pytest.mark.parametrize("case", ROPES, ids=lambda c: "%dx%d-%s-%d" % (c[0], c[1], "+".join(map(str, c[2])), c[3]))
def test_rope(case, layout):
    heads, hd, dims, rows = case
    g = torch.Generator(device=DEV).manual_seed(rows + hd)
    w = heads * hd
    r = dlo.make_rope(heads=heads, head_dim=hd, layout=layout, ldx=w + 24, ldy=w + 8, amp=1.25,
                      axes=[dict(dim=d, theta=100.0 * 10 ** i) for i, d in enumerate(dims)])
    steps = torch.from_numpy(dlo.dlo_rope_steps(r)).to(DEV)
    x = torch.randn((rows, w + 24), generator=g, device=DEV).to(torch.bfloat16)
    positions = torch.randint(-3000, 100000, (rows, len(dims)), generator=g, device=DEV, dtype=torch.int32)
    positions[0] = torch.iinfo(torch.int32).max
    positions[-1] = torch.iinfo(torch.int32).min
    y = torch.full((rows, w + 8), KEEP, dtype=torch.bfloat16, device=DEV)
    dlo.dlo_op_rope_fwd(r, x.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, y.data_ptr(), stream())
    want, size = rope_reference(r, x[:, :w], positions)
    within(y[:, :w], want, U * want.abs() + 2.0 ** -20 * size + 1e-30, "y")
    assert bool((y[:, w:] == KEEP).all())
    back = torch.full((rows, w + 24), KEEP, dtype=torch.bfloat16, device=DEV)
    dlo.dlo_op_rope_bwd(r, y.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, back.data_ptr(), stream())
    want, size = rope_reference(r, y[:, :w], positions, back=True)
    within(back[:, :w], want, U * want.abs() + 2.0 ** -20 * size + 1e-30, "dx")
    assert bool((back[:, w:] == KEEP).all())
    # in place: the same bits
    r.ldy = r.ldx
    z = x.clone()
    dlo.dlo_op_rope_fwd(r, z.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, z.data_ptr(), stream())
    assert torch.equal(z[:, :w], y[:, :w]) and torch.equal(z[:, w:], x[:, w:])
    r.ldy = w + 8
    z = y.clone()
    r.ldx = r.ldy
    dlo.dlo_op_rope_bwd(r, z.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, z.data_ptr(), stream())
    assert torch.equal(z[:, :w], back[:, :w])


@pytest.mark.parametrize("scaling", [dlo.ROPE_PLAIN, dlo.ROPE_LINEAR, dlo.ROPE_BASE, dlo.ROPE_BY_TURNS, dlo.ROPE_BY_INDEX])
def test_rope_scalings_far_out(scaling):
    heads, hd, rows = 4, 64, 257
    r = dlo.make_rope(heads=heads, head_dim=hd, ldx=256, ldy=256, layout=dlo.ROPE_HALF,
                      axes=[dict(dim=hd, scaling=scaling, factor=16.0, length=8192.0)])
    steps = torch.from_numpy(dlo.dlo_rope_steps(r)).to(DEV)
    x = torch.randn((rows, 256), device=DEV).to(torch.bfloat16)
    positions = (1000003 * torch.arange(rows, device=DEV, dtype=torch.int32))[:, None].contiguous()
    y = torch.empty_like(x)
    dlo.dlo_op_rope_fwd(r, x.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, y.data_ptr(), stream())
    want, size = rope_reference(r, x, positions)
    within(y, want, U * want.abs() + 2.0 ** -20 * size + 1e-30, "y")


def test_rope_inside_fused_rows():
    """q and k of fused q | k | v rows in one call, in place; v stays."""
    H, G, hd, rows = 6, 2, 64, 100
    ld = (H + 2 * G) * hd
    r = dlo.make_rope(heads=H + G, head_dim=hd, ldx=ld, ldy=ld, axes=[dict(dim=hd)])
    steps = torch.from_numpy(dlo.dlo_rope_steps(r)).to(DEV)
    x = torch.randn((rows, ld), device=DEV).to(torch.bfloat16)
    positions = torch.arange(rows, device=DEV, dtype=torch.int32)
    y = x.clone()
    dlo.dlo_op_rope_fwd(r, y.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, y.data_ptr(), stream())
    want, size = rope_reference(r, x[:, :(H + G) * hd], positions[:, None])
    within(y[:, :(H + G) * hd], want, U * want.abs() + 2.0 ** -20 * size + 1e-30, "y")
    assert torch.equal(y[:, (H + G) * hd:], x[:, (H + G) * hd:])
