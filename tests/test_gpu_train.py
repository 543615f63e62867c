"""Training ops (attention, LayerNorm, RMSNorm and their backward passes)
against plain forms in 64 bits.

Attention bounds are element-wise and follow from the roundings: u = 2^-8 is
half a bf16 step relative to the value.  With P, dS rounded to bf16 before their
products and O as given (rounded):
  |O err|  <= u (sum_j p |v| + |o|)
  |dV err| <= u (sum_i p |do| + |dv|)
  |D err|  <= u sum_d |do o|  =: e_i,   |dS err| <= u |dS| + p e
  |dQ err| <= (sum_j (u |dS| + p e) |k|) / sqrt(hd) + u |dQ|, and dK likewise
plus what fp32 adds: a score of magnitude s is off by ~2^-22 (sum_d |q k|) / sqrt(hd)
<= f relative in p, with f = 2^-18 for |q|.|k| / sqrt(hd) <= 16, and dP by 2^-20
sum_d |do v|.  u is taken 1% larger for products of two roundings.
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


@pytest.fixture(autouse=True)
def float32_by_default():
    """Another test module of the same process may have set another default."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return None if t is None else t.data_ptr()


def bytes_(n):
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")     # NaN where read unwritten


class Problem:
    """One attention problem with fused or separate rows and a 64-bit reference."""

    def __init__(self, B, H, G, hd, nq, nk, cb=0, q_lens=None, k_lens=None, seed=0, pad=0, fused=True, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * nq + 13 * nk + hd)
        self.c = (B, H, G, hd, nq, nk, cb)
        self.q_lens = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
        self.k_lens = None if k_lens is None else torch.tensor(k_lens, dtype=torch.int32, device="cuda")
        self.ql = [nq] * B if q_lens is None else [min(max(x, 0), nq) for x in q_lens]
        self.kl = [nk] * B if k_lens is None else [min(max(x, 0), nk) for x in k_lens]

        def rnd(shape, s=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * s).to(torch.bfloat16)

        if fused and nq == nk:
            rows = rnd((B, nq, (H + 2 * G) * hd + pad), scale)
            self.q, self.k, self.v = rows[..., :H * hd], rows[..., H * hd:(H + G) * hd], rows[..., (H + G) * hd:(H + 2 * G) * hd]
        else:
            self.q = rnd((B, nq, H * hd + pad), scale)[..., :H * hd]
            kv = rnd((B, nk, 2 * G * hd + pad), scale)
            self.k, self.v = kv[..., :G * hd], kv[..., G * hd:2 * G * hd]
        self.do = rnd((B, nq, H * hd + pad), 0.1)[..., :H * hd]
        for b in range(B):                          # what lies behind the sequences is never used
            for t, n in ((self.q, self.ql), (self.do, self.ql), (self.k, self.kl), (self.v, self.kl)):
                t[b, n[b]:] = NAN
        self.o = torch.full((B, nq, H * hd + pad), NAN, dtype=torch.bfloat16, device="cuda")[..., :H * hd]
        self.lse = torch.full((B, H, nq), NAN, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def desc(self, grads=()):
        B, H, G, hd, nq, nk, cb = self.c
        ld = dict(zip(("lddq", "lddk", "lddv"), (t.stride(1) for t in grads)))
        return dlo.make_attn(batch=B, heads=H, kv_heads=G, head_dim=hd, nq=nq, nk=nk, causal_block=cb,
                             ldq=self.q.stride(1), ldk=self.k.stride(1), ldv=self.v.stride(1), ldo=self.o.stride(1),
                             lddo=self.do.stride(1), q_lens=ptr(self.q_lens), k_lens=ptr(self.k_lens), **ld)

    def forward(self, ws=None):
        a = self.desc()
        ws = bytes_(dlo.dlo_attention_fwd_workspace_bytes(a)) if ws is None else ws
        dlo.dlo_op_attention_fwd(a, self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.o.data_ptr(),
                                 self.lse.data_ptr(), ws.data_ptr(), ws.numel(), self.err.data_ptr(), stream())
        return ws

    def grads(self, pad=0):
        B, H, G, hd, nq, nk, _ = self.c
        return [torch.full((B, n, w * hd + pad), 3.5, dtype=torch.bfloat16, device="cuda")[..., :w * hd]
                for n, w in ((nq, H), (nk, G), (nk, G))]

    def backward(self, grads, ws=None):
        a = self.desc(grads)
        ws = bytes_(dlo.dlo_attention_bwd_workspace_bytes(a)) if ws is None else ws
        dlo.dlo_op_attention_bwd(a, self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.o.data_ptr(),
                                 self.lse.data_ptr(), self.do.data_ptr(), *(t.data_ptr() for t in grads),
                                 ws.data_ptr(), ws.numel(), self.err.data_ptr(), stream())
        return ws

    def reference(self):
        """O, lse, dQ, dK, dV in 64 bits and their error bounds."""
        B, H, G, hd, nq, nk, cb = self.c
        z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")                    # noqa: E731
        out = {k: z(B, nq, H, hd) for k in ("o", "dq", "o_b", "dq_b")}
        out |= {k: z(B, nk, G, hd) for k in ("dk", "dv", "dk_b", "dv_b")}
        out["lse"] = torch.full((B, H, nq), -math.inf, dtype=torch.float64, device="cuda")
        i = torch.arange(nq, device="cuda")[:, None] + nk - nq
        j = torch.arange(nk, device="cuda")[None]
        for b in range(B):
            see = (torch.arange(nq, device="cuda")[:, None] < self.ql[b]) & (j < self.kl[b])
            if cb:
                see = see & (i >= 0) & (torch.div(i, cb, rounding_mode="floor") >= torch.div(j, cb, rounding_mode="floor"))
            any_ = see.any(1)
            for h in range(H):
                g = h // (H // G)
                clean = lambda t, n, w: torch.nan_to_num(t[b, :, w * hd:(w + 1) * hd].double()) * (torch.arange(t.shape[1], device="cuda") < n[b])[:, None]   # noqa: E731
                q, do = clean(self.q, self.ql, h), clean(self.do, self.ql, h)
                k, v = clean(self.k, self.kl, g), clean(self.v, self.kl, g)
                s = (q @ k.T / math.sqrt(hd)).masked_fill(~see, -math.inf)
                lse = torch.where(any_, torch.logsumexp(s, 1), -math.inf)
                p = torch.where(see, torch.exp(s - torch.where(any_, lse, 0.0)[:, None]), 0.0)
                o = p @ v
                out["lse"][b, h] = lse
                out["o"][b, :, h] = o
                out["o_b"][b, :, h] = (U + F) * (p @ v.abs()) + U * o.abs() + 1e-30
                dv = p.T @ do
                out["dv"][b, :, g] += dv
                out["dv_b"][b, :, g] += (U + F) * (p.T @ do.abs())
                dp = do @ v.T
                D = (do * o).sum(1, keepdim=True)
                # D from the O that the forward left: its whole error, not one rounding only
                e = (do.abs() * out["o_b"][b, :, h]).sum(1, keepdim=True)
                ds = p * (dp - D)
                ds_b = (U + F) * ds.abs() + p * (e + 2.0 ** -20 * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True)))
                out["dq"][b, :, h] = ds @ k / math.sqrt(hd)
                out["dq_b"][b, :, h] = ds_b @ k.abs() / math.sqrt(hd) + U * out["dq"][b, :, h].abs() + 1e-30
                out["dk"][b, :, g] += ds.T @ q / math.sqrt(hd)
                out["dk_b"][b, :, g] += ds_b.T @ q.abs() / math.sqrt(hd)
        for x in ("dk", "dv"):
            out[x + "_b"] += U * out[x].abs() + 1e-30
        return out

    def check(self, ref, grads=None):
        B, H, G, hd, nq, nk, _ = self.c
        assert int(self.err.item()) == 0
        within(self.o.reshape(B, nq, H, hd), ref["o"], ref["o_b"], "O")
        empty = ref["lse"] == -math.inf
        assert torch.equal(self.lse == -math.inf, empty), "empty rows"
        d = (self.lse.double() - ref["lse"])[~empty]
        # scores of magnitude <= 16 in fp32 products, exp and log within a few ulp
        assert d.numel() == 0 or float(d.abs().max()) <= 1e-5
        if grads is not None:
            within(grads[0].reshape(B, nq, H, hd), ref["dq"], ref["dq_b"], "dQ")
            within(grads[1].reshape(B, nk, G, hd), ref["dk"], ref["dk_b"], "dK")
            within(grads[2].reshape(B, nk, G, hd), ref["dv"], ref["dv_b"], "dV")


def within(y, ref, bound, name):
    d = (y.double() - ref).abs()
    assert torch.isfinite(d).all(), f"{name}: not finite"
    over = float((d / bound).max())
    assert over <= 1, f"{name}: error {over:.3f} of its bound"


CASES = [
    # B, H, G, hd, nq, nk, causal block, q_lens, k_lens
    (1, 1, 1, 8, 1, 1, 0, None, None),
    (1, 1, 1, 64, 128, 128, 0, None, None),
    (1, 2, 2, 128, 128, 256, 0, None, None),
    (1, 2, 2, 128, 300, 300, 0, None, None),
    (2, 4, 4, 72, 257, 257, 0, None, None),
    (1, 4, 4, 64, 1, 300, 0, None, None),
    (1, 2, 2, 64, 300, 1, 0, None, None),
    (2, 6, 2, 64, 130, 259, 0, None, None),
    (1, 8, 1, 40, 131, 70, 0, None, None),
    (2, 4, 2, 72, 300, 140, 0, [300, 129], [1, 128]),
    (3, 4, 2, 128, 260, 260, 0, [0, 260, 131], [260, 0, 5]),
    (3, 2, 1, 80, 200, 385, 0, [128, 127, 129], [256, 129, 384]),
    (2, 2, 2, 16, 260, 260, 1, None, None),
    (2, 4, 1, 64, 300, 300, 1, [300, 170], [300, 170]),
    (1, 2, 2, 96, 150, 400, 1, None, None),
    (1, 2, 2, 112, 400, 150, 1, None, None),          # the first 250 queries see nothing
    (1, 2, 2, 128, 600, 600, 100, None, None),
    (2, 2, 2, 72, 513, 513, 170, [513, 300], [500, 301]),
    (1, 2, 2, 88, 260, 260, 1 << 30, None, None),     # one block: every key
    (1, 3, 3, 64, 700, 130, 7, None, [100]),
    (2, 2, 2, 64, 130, 130, 0, [200, -3], [1 << 30, 50]),     # lengths out of range are taken into it
    (1, 2, 1, 64, 5, 4100, 0, None, [4001]),          # few queries: the keys are split
    (2, 2, 2, 128, 17, 5000, 1, [17, 9], [5000, 300]),
    (1, 2, 2, 64, 2500, 100, 0, None, None),          # few keys: their gradients are split over the queries
    (2, 4, 2, 72, 1500, 1500, 1, [1500, 900], [1500, 900]),   # causal: likewise
    (2, 8, 2, 128, 33, 1300, 0, [33, 7], [1300, 515]),        # heads of a group share query tiles
    (1, 24, 2, 64, 10, 700, 1, None, None),           # groups of 12: four heads a tile
    (2, 16, 1, 40, 1, 260, 0, [1, 0], None),
    (1, 8, 1, 72, 100, 90, 30, None, [50]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:7])) + ("-lens" if c[7] or c[8] else ""))
def test_attention_forward_and_backward(case):
    p = Problem(*case)
    p.forward()
    grads = p.grads()
    p.backward(grads)
    torch.cuda.synchronize()
    p.check(p.reference(), grads)


def _small(seed=3):
    return Problem(2, 4, 2, 64, 300, 300, 50, [300, 190], [280, 300], seed=seed)


def test_attention_strides_and_rows_around_are_left_alone():
    p = Problem(2, 4, 2, 72, 140, 200, 0, None, [200, 77], pad=24)
    p.forward()
    grads = [torch.full((t.shape[0], t.shape[1], t.shape[2] + 40), 3.5, dtype=torch.bfloat16, device="cuda") for t in p.grads()]
    views = [t[..., 16:t.shape[2] - 24] for t in grads]
    p.backward(views)
    torch.cuda.synchronize()
    p.check(p.reference(), views)
    for t in grads:
        assert (t[..., :16] == 3.5).all() and (t[..., t.shape[2] - 24:] == 3.5).all()


def test_attention_gradients_into_one_fused_buffer():
    B, H, G, hd, n = 2, 4, 2, 64, 200
    p = Problem(B, H, G, hd, n, n, 1)
    p.forward()
    rows = torch.empty((B, n, (H + 2 * G) * hd), dtype=torch.bfloat16, device="cuda")
    views = rows.split([H * hd, G * hd, G * hd], dim=-1)
    p.backward(views)
    torch.cuda.synchronize()
    p.check(p.reference(), views)


def test_attention_same_bits_every_time_on_another_stream_and_from_a_graph():
    p = _small()
    a, b = p.grads(), p.grads()
    p.forward()
    p.backward(a)
    torch.cuda.synchronize()
    o, lse = p.o.clone(), p.lse.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ws = p.forward()
        wb = p.backward(b)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(p.o)) and torch.equal(lse, p.lse)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.forward(ws)
        p.backward(b, wb)
    for seed in (5, 6):                      # new inputs in the same buffers, lengths among them
        other = _small(seed)
        for x, y in ((p.q, other.q), (p.k, other.k), (p.v, other.v), (p.do, other.do)):
            x.copy_(y)
        g.replay()
        fresh = other.grads()
        other.forward()
        other.backward(fresh)
        torch.cuda.synchronize()
        assert torch.equal(p.lse, other.lse) and torch.equal(p.o, other.o)
        assert all(torch.equal(x, y) for x, y in zip(b, fresh))


def test_attention_two_calls_at_once_with_their_own_workspaces():
    p, q = _small(1), _small(2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    gp, gq = p.grads(), q.grads()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(s1):
            p.forward()
            kp = p.backward(gp)
        with torch.cuda.stream(s2):
            q.forward()
            kq = q.backward(gq)
        torch.cuda.synchronize()
    p.check(p.reference(), gp)
    q.check(q.reference(), gq)
    del kp, kq


def test_attention_backward_agrees_with_differences():
    """<dQ, u> + <dK, v> + <dV, w> against the central difference of <O, dO> in 64 bits along (u, v, w)."""
    B, H, G, hd, n, m = 1, 2, 1, 64, 140, 150
    p = Problem(B, H, G, hd, n, m, 0, None, [130])
    p.forward()
    grads = p.grads()
    p.backward(grads)
    torch.cuda.synchronize()
    ref = p.reference()
    g = torch.Generator(device="cuda").manual_seed(9)
    saved = [t.clone() for t in (p.q, p.k, p.v)]
    clean = [torch.nan_to_num(t.double()) for t in saved]
    dirs = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in clean]
    dirs[1][:, 130:] = 0
    dirs[2][:, 130:] = 0

    def loss(e):
        q, k, v = (x + e * d for x, d in zip(clean, dirs))
        total = 0.0
        for h in range(H):
            s = q[0, :, h * hd:(h + 1) * hd] @ k[0, :130].T / math.sqrt(hd)
            total = total + (torch.softmax(s, 1) @ v[0, :130] * p.do[0, :, h * hd:(h + 1) * hd].double()).sum()
        return float(total)

    e = 1e-4
    want = (loss(e) - loss(-e)) / (2 * e)
    got = sum(float((t.double() * d).sum()) for t, d in zip(grads, dirs))
    bound = sum(float((ref[x + "_b"].reshape(d.shape) * d.abs()).sum()) for x, d in zip(("dq", "dk", "dv"), dirs))
    assert abs(got - want) <= bound + 1e-6 * abs(want)
    # the bound is a worst case; the sum over thousands of independent roundings stays far inside
    assert abs(got - want) <= 0.02 * abs(want) + 0.05 * bound


# ------------------------------------------------------------------ norms

NORM_F = 2.0 ** -18      # fp32 row sums (<= 20480 terms in trees and chains of <= 160), rsqrt, products


def _ln_reference(x, dy, gain, add, dres, rpb):
    x, dy = x.double(), dy.double()
    D = x.shape[1]
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + 1e-6)
    xh = (x - mean) * rstd
    g = dy * gain
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2) + dres
    size = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + (xh.abs() + 1) * (g * xh).abs().mean(1, keepdim=True)) + abs(dres)
    y = xh * gain + add
    groups = [slice(i, min(i + rpb, x.shape[0])) for i in range(0, x.shape[0], rpb)]
    s1 = torch.stack([dy[r].sum(0) for r in groups])
    s2 = torch.stack([(dy * xh)[r].sum(0) for r in groups])
    # xh itself is off by up to NORM_F of the row's scale
    b1 = torch.stack([dy[r].abs().sum(0) for r in groups])
    b2 = torch.stack([(dy.abs() * (xh.abs() + x.abs().amax(1, keepdim=True) * rstd))[r].sum(0) for r in groups])
    span = x.abs().amax(1, keepdim=True) * rstd
    return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0], dx=dx, s1=s1, s2=s2,
                y_b=U * y.abs() + NORM_F * (span + 1) * abs(gain) + NORM_F * abs(add) + 1e-30,
                dx_b=NORM_F * (1 + span) * size + 1e-30, s1_b=NORM_F * b1 + 1e-30, s2_b=NORM_F * b2 + 1e-30)


@pytest.mark.parametrize("form", ["mod", "affine", "plain"])
@pytest.mark.parametrize("rows,D,rpb", [(1, 4, 1), (3, 64, 2), (7, 132, 7), (300, 1152, 150), (260, 1284, 100), (97, 2564, 50),
                                        (2048, 1152, 1024), (4096, 1152, 1024), (333, 5120, 333), (20, 10244, 9), (5, 20480, 2), (700, 256, 1),
                                        (5000, 68, 1700)])
def test_layernorm_forward_and_backward(form, rows, D, rpb):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    rnd = lambda *s, k=1.0: torch.randn(s, generator=g, device="cuda") * k                    # noqa: E731
    nb = (rows + rpb - 1) // rpb
    x = rnd(rows, D) * (0.5 + torch.rand((rows, 1), generator=g, device="cuda")) + 0.3
    dy = rnd(rows, D, k=0.1).to(torch.bfloat16)
    dres = rnd(rows, D, k=0.1)
    mod = rnd(nb, 3 * D + 4, k=0.3)                  # shift | scale | something else
    w, b = (1 + rnd(D, k=0.1)).to(torch.bfloat16), rnd(D, k=0.1).to(torch.bfloat16)
    batch = torch.arange(rows, device="cuda") // rpb
    shift = scale = wp = bp = None
    gain, add, group = 1.0, 0.0, rows
    if form == "mod":
        shift, scale = mod.data_ptr(), mod[:, D:].data_ptr()
        gain, add, group = 1 + mod[batch, D:2 * D].double(), mod[batch, :D].double(), rpb
    elif form == "affine":
        wp, bp = w.data_ptr(), b.data_ptr()
        gain, add = w.double(), b.double()
    y = torch.full((rows, D), NAN, dtype=torch.bfloat16, device="cuda")
    mean, rstd = torch.full((rows,), NAN, device="cuda"), torch.full((rows,), NAN, device="cuda")
    dlo.dlo_op_layernorm_fwd(x.data_ptr(), rows, D, rpb, shift, scale, mod.stride(0), wp, bp, 1e-6, y.data_ptr(),
                             mean.data_ptr(), rstd.data_ptr(), stream())
    gain_t = gain if torch.is_tensor(gain) else torch.ones((), device="cuda", dtype=torch.float64)
    add_t = add if torch.is_tensor(add) else torch.zeros((), device="cuda", dtype=torch.float64)
    r = _ln_reference(x, dy, gain_t, add_t, dres.double(), group)
    within(y, r["y"], r["y_b"], "y")
    within(mean, r["mean"], NORM_F * x.double().abs().mean(1) + 1e-30, "mean")
    within(rstd, r["rstd"], NORM_F * r["rstd"] * (1 + r["rstd"] * x.double().abs().amax(1)), "rstd")
    ws = bytes_(dlo.dlo_layernorm_bwd_workspace_bytes(rows, D, rpb))
    dx = torch.full((rows, D), NAN, device="cuda")
    dmod = torch.full((nb, 3 * D + 4), 7.0, device="cuda")
    dw, db = torch.full((D,), NAN, device="cuda"), torch.full((D,), NAN, device="cuda")
    # the scale's gradient lies before the shift's here: their order is free
    p1, p2 = {"mod": (dmod[:, D:], dmod), "affine": (db, dw), "plain": (None, None)}[form]

    def backward(dres_t, dx_t, q1=p1, q2=p2):
        dlo.dlo_op_layernorm_bwd(dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, D, rpb, scale,
                                 mod.stride(0), wp, ptr(dres_t), dx_t.data_ptr(), ptr(q1), ptr(q2), dmod.stride(0),
                                 ws.data_ptr(), ws.numel(), stream())

    backward(dres, dx)
    within(dx, r["dx"], r["dx_b"], "dx")
    if form == "mod":
        within(dmod[:, D:2 * D], r["s1"], r["s1_b"], "dshift")
        within(dmod[:, :D], r["s2"], r["s2_b"], "dscale")
        assert (dmod[:, 2 * D:] == 7.0).all()
    elif form == "affine":
        within(db[None], r["s1"], r["s1_b"], "db")
        within(dw[None], r["s2"], r["s2_b"], "dw")
    again, keep = dres.clone(), dx.clone()
    backward(again, again)                           # in place over the residual's gradient
    assert torch.equal(again, keep)
    backward(None, dx, None, None)                   # frozen parameters, no residual
    within(dx, r["dx"] - dres.double(), r["dx_b"], "dx without dres")


@pytest.mark.parametrize("rows,D,pad", [(1, 8, 0), (5, 64, 16), (300, 1152, 2304), (8192 + 3, 256, 0), (1900, 4104, 0), (77, 1288, 8), (130, 2568, 0),
                                        (300, 5120, 10240), (33, 7000, 0), (9, 20480, 8)])
def test_rmsnorm_forward_and_backward(rows, D, pad):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    rnd = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(torch.bfloat16)      # noqa: E731
    ld = D + pad
    x, dy, w = rnd(rows, ld)[:, pad:], rnd(rows, ld, k=0.1)[:, pad:], 1 + rnd(D, k=0.1)
    y = torch.full((rows, D), NAN, dtype=torch.bfloat16, device="cuda")
    rstd = torch.full((rows,), NAN, device="cuda")
    dlo.dlo_op_rmsnorm_fwd(x.data_ptr(), ld, rows, D, w.data_ptr(), 1e-6, y.data_ptr(), D, rstd.data_ptr(), stream())
    X, DY, W = x.double(), dy.double(), w.double()
    r = 1 / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-6)
    xh = X * r
    within(y, xh * W, (U + NORM_F) * (xh * W).abs() + 1e-30, "y")
    within(rstd, r[:, 0], NORM_F * r[:, 0], "rstd")
    gg = DY * W
    c = (gg * xh).mean(1, keepdim=True)
    want = r * (gg - xh * c)
    bound = U * want.abs() + NORM_F * r * (gg.abs() + xh.abs() * (gg * xh).abs().mean(1, keepdim=True)) + 1e-30
    ws = bytes_(dlo.dlo_rmsnorm_bwd_workspace_bytes(rows, D))
    whole = torch.full((rows, ld), 2.5, dtype=torch.bfloat16, device="cuda")
    dx, dw = whole[:, pad:], torch.full((D,), NAN, device="cuda")

    def backward(dy_t, dx_t, dw_t=dw):
        dlo.dlo_op_rmsnorm_bwd(dy_t.data_ptr(), ld, x.data_ptr(), ld, w.data_ptr(), rstd.data_ptr(), rows, D,
                               dx_t.data_ptr(), ld, ptr(dw_t), ws.data_ptr(), ws.numel(), stream())

    backward(dy, dx)
    within(dx, want, bound, "dx")
    within(dw, (DY * xh).sum(0), NORM_F * (DY * xh).abs().sum(0) + 1e-30, "dw")
    assert (whole[:, :pad] == 2.5).all()
    keep, same = dx.clone(), torch.full((D,), NAN, device="cuda")
    inplace = dy.clone()[:, :D] if not pad else torch.cat([torch.zeros_like(whole[:, :pad]), dy], 1)[:, pad:]
    backward(inplace, inplace, same)                 # in place, and the weight's gradient all the same
    assert torch.equal(inplace, keep)
    within(same, (DY * xh).sum(0), NORM_F * (DY * xh).abs().sum(0) + 1e-30, "dw in place")
    backward(dy, dy, None)
    assert torch.equal(dy, keep)


def test_norm_backward_from_a_graph_and_on_another_stream():
    rows, D = 300, 1152
    g = torch.Generator(device="cuda").manual_seed(0)
    x, dy = torch.randn((rows, D), generator=g, device="cuda"), torch.randn((rows, D), generator=g, device="cuda").to(torch.bfloat16)
    w, b = torch.ones(D, dtype=torch.bfloat16, device="cuda"), torch.zeros(D, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = torch.empty_like(dy), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = bytes_(dlo.dlo_layernorm_bwd_workspace_bytes(rows, D, rows))
    out = [torch.empty((rows, D), device="cuda"), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]

    def both():
        dlo.dlo_op_layernorm_fwd(x.data_ptr(), rows, D, rows, None, None, 0, w.data_ptr(), b.data_ptr(), 1e-6, y.data_ptr(),
                                 mean.data_ptr(), rstd.data_ptr(), stream())
        dlo.dlo_op_layernorm_bwd(dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, D, rows, None, 0,
                                 w.data_ptr(), None, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), 0, ws.data_ptr(),
                                 ws.numel(), stream())

    both()
    torch.cuda.synchronize()
    keep = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in out:
        t.fill_(NAN)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(out, keep))
    x.mul_(1.5)
    graph.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = [t.clone() for t in out]
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(out, keep))


# ------------------------------------------------------------------ together

def test_gradient_through_the_attention_half_of_a_video_block():
    """x -> LayerNorm (modulated) -> q|k|v linear -> RMSNorm of q and k -> attention,
    and the gradient back to x, the modulation and the norms' weights, against
    autograd in 64 bits.  About ten bf16 roundings lie on the way (h, qkv, q and
    k, P, O, dS, dqkv twice, dh), each at most 2^-8 relative; a quarter of
    their sum over the whole tensor leaves room for their random signs only."""
    B, N, H, hd = 2, 200, 4, 64
    D = H * hd
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, k=1.0: torch.randn(s, generator=g, device="cuda") * k                    # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)                                                       # noqa: E731
    x, mod = rnd(B, N, D), rnd(B, 2 * D, k=0.3)
    W, bias = bf(rnd(3 * D, D, k=D ** -0.5)), bf(rnd(3 * D, k=0.1))
    wq, wk = bf(1 + rnd(D, k=0.1)), bf(1 + rnd(D, k=0.1))
    do = bf(rnd(B, N, D, k=0.1))
    k_lens = torch.tensor([N, 150], dtype=torch.int32, device="cuda")
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")                   # noqa: E731
    f32, s, R = torch.float32, stream(), B * N
    h, mean, rstd, qkv, qk, rq, rk = e(R, D), e(R, t=f32), e(R, t=f32), e(R, 3 * D), e(R, 2 * D), e(R, t=f32), e(R, t=f32)
    o, lse, err = e(B, N, D), e(B, H, N, t=f32), torch.zeros(1, dtype=torch.int32, device="cuda")
    dlo.dlo_op_layernorm_fwd(x.data_ptr(), R, D, N, mod.data_ptr(), mod[:, D:].data_ptr(), 2 * D, None, None, 1e-6, h.data_ptr(),
                             mean.data_ptr(), rstd.data_ptr(), s)
    dlo.dlo_op_gemm(h.data_ptr(), W.data_ptr(), dlo.DT_BF16, None, 0, bias.data_ptr(), R, 3 * D, D, dlo.EPI_BIAS, qkv.data_ptr(),
                    3 * D, None, 0, 1, err.data_ptr(), s)
    for c, w, r in ((0, wq, rq), (1, wk, rk)):
        dlo.dlo_op_rmsnorm_fwd(qkv[:, c * D:].data_ptr(), 3 * D, R, D, w.data_ptr(), 1e-6, qk[:, c * D:].data_ptr(), 2 * D,
                               r.data_ptr(), s)
    a = dlo.make_attn(batch=B, heads=H, head_dim=hd, nq=N, nk=N, causal_block=20, ldq=2 * D, ldk=2 * D, ldv=3 * D, ldo=D,
                      lddq=3 * D, lddk=3 * D, lddv=3 * D, lddo=D, k_lens=k_lens.data_ptr())
    ws = bytes_(max(dlo.dlo_attention_fwd_workspace_bytes(a), dlo.dlo_attention_bwd_workspace_bytes(a),
                    dlo.dlo_rmsnorm_bwd_workspace_bytes(R, D), dlo.dlo_layernorm_bwd_workspace_bytes(R, D, N)))
    v = qkv[:, 2 * D:]
    dlo.dlo_op_attention_fwd(a, qk.data_ptr(), qk[:, D:].data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                             ws.numel(), err.data_ptr(), s)
    dqkv, dwq, dwk, dh, dx, dmod = e(R, 3 * D), e(D, t=f32), e(D, t=f32), e(R, D), e(B, N, D, t=f32), e(B, 2 * D, t=f32)
    dlo.dlo_op_attention_bwd(a, qk.data_ptr(), qk[:, D:].data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                             dqkv.data_ptr(), dqkv[:, D:].data_ptr(), dqkv[:, 2 * D:].data_ptr(), ws.data_ptr(), ws.numel(),
                             err.data_ptr(), s)
    for c, w, r, dw in ((0, wq, rq, dwq), (1, wk, rk, dwk)):
        t = dqkv[:, c * D:]
        dlo.dlo_op_rmsnorm_bwd(t.data_ptr(), 3 * D, qkv[:, c * D:].data_ptr(), 3 * D, w.data_ptr(), r.data_ptr(), R, D,
                               t.data_ptr(), 3 * D, dw.data_ptr(), ws.data_ptr(), ws.numel(), s)
    Wt = W.T.contiguous()
    dlo.dlo_op_gemm(dqkv.data_ptr(), Wt.data_ptr(), dlo.DT_BF16, None, 0, None, R, D, 3 * D, dlo.EPI_BIAS, dh.data_ptr(), D,
                    None, 0, 1, err.data_ptr(), s)
    dlo.dlo_op_layernorm_bwd(dh.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), R, D, N, mod[:, D:].data_ptr(), 2 * D,
                             None, None, dx.data_ptr(), dmod.data_ptr(), dmod[:, D:].data_ptr(), 2 * D, ws.data_ptr(),
                             ws.numel(), s)
    torch.cuda.synchronize()
    assert int(err.item()) == 0

    X, M, WQ, WK = (t.double().requires_grad_() for t in (x, mod, wq, wk))
    mu = X.mean(-1, keepdim=True)
    xh = (X - mu) / torch.sqrt(((X - mu) ** 2).mean(-1, keepdim=True) + 1e-6)
    Y = (xh * (1 + M[:, None, D:]) + M[:, None, :D]) @ W.double().T + bias.double()
    rms = lambda t, w: t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w              # noqa: E731
    split = lambda t: t.reshape(B, N, H, hd).transpose(1, 2)                                  # noqa: E731
    Q, K, V = split(rms(Y[..., :D], WQ)), split(rms(Y[..., D:2 * D], WK)), split(Y[..., 2 * D:])
    i = torch.arange(N, device="cuda")
    see = (i[:, None] // 20 >= i[None] // 20)[None, None] & (i[None, :] < k_lens[:, None])[:, None, None]
    O = (torch.softmax((Q @ K.transpose(-1, -2) / math.sqrt(hd)).masked_fill(~see, -math.inf), -1) @ V).transpose(1, 2).reshape(B, N, D)
    O.backward(do.double())
    for name, got, want in (("o", o, O.detach()), ("dx", dx, X.grad), ("dmod", dmod, M.grad), ("dwq", dwq, WQ.grad), ("dwk", dwk, WK.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 10 * 2.0 ** -8, f"{name}: {rel:.3e}"


@pytest.mark.parametrize("case", [(2, 16, 16, 72, 1024, 1024), (2, 10, 10, 128, 2000, 512), (2, 8, 2, 64, 1500, 1500, 1)],
                         ids=lambda c: "x".join(map(str, c)))
def test_attention_keeps_its_bits_over_many_calls(case):
    """A wait that misses a phase, or an arrival counted for the wrong one, shows up rarely:
    as other bits, or as the error word of a wait that ran out."""
    p = Problem(*case)
    grads = p.grads()
    wf, wb = p.forward(), p.backward(grads)
    torch.cuda.synchronize()
    keep = [t.clone() for t in (p.o, p.lse, *grads)]
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        p.forward(wf)
        p.backward(grads, wb)
        if i % 4 == 0:
            for a, b in zip(keep, (p.o, p.lse, *grads)):
                differ += (a != b).sum()
    assert int(differ.item()) == 0 and int(p.err.item()) == 0


@pytest.mark.parametrize("case", [(1, 4, 4, 64, 256, 256), (2, 8, 8, 128, 300, 77), (2, 16, 16, 72, 1024, 1024), (2, 16, 4, 64, 40, 1500)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_attention_backward_reads_what_was_written_just_before(case, graph):
    """Inputs and lengths change in place right before each call, nothing waits on the host:
    every launch of the call has to see the new ones, whichever starts early."""
    nq, nk = case[4:6]
    lens = [None] * 3 if case[0] == 1 else [([nq, nq - 19], [nk - 5, nk]), ([nq - 33, nq], [nk, nk - 40]), ([nq - 1, 1], [1, nk - 1])]
    sets = [Problem(*case, 0, *(lens[i] or (None, None)), seed=50 + i, fused=False) for i in range(3)]
    want = []
    for s in sets:
        s.forward()
        want.append(s.grads())
        torch.cuda.synchronize()
        s.backward(want[-1])
        torch.cuda.synchronize()
    names = ("q", "k", "v", "do", "o", "lse") + (() if lens[0] is None else ("q_lens", "k_lens"))
    p = Problem(*case, 0, *(lens[0] or (None, None)), seed=50, fused=False)
    grads = p.grads()
    ws = bytes_(dlo.dlo_attention_bwd_workspace_bytes(p.desc(grads)))
    differ = torch.zeros((), dtype=torch.int64, device="cuda")

    def one_round():
        for s, w in zip(sets, want):
            for n in names:
                getattr(p, n).copy_(getattr(s, n))
            p.backward(grads, ws)
            for a, b in zip(grads, w):
                differ.add_((a != b).sum())

    one_round()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one_round()
        one_round = g.replay
    for _ in range(30):
        one_round()
    assert int(differ.item()) == 0 and int(p.err.item()) == 0


@pytest.mark.parametrize("nq,nk,cb,klen", [(40, 2, 0, None), (130, 300, 0, 3), (64, 64, 1, None), (257, 128, 0, 100), (100, 100, 10, 77)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_gradients_of_few_keys_do_not_carry_the_rounding_of_o(nq, nk, cb, klen, hd):
    """Rows that lie in one key tile: D is the sum of P dP, off by what fp32 makes of P (f, relative)
    and dP (2^-20 of |do||v|), so dS is right to f |dS| + P (f + 2^-20) (|do||v| + sum P |do||v|)
    before its rounding.  With D from a bf16 O, dQ misses this bound."""
    H = 3
    p = Problem(1, H, H, hd, nq, nk, cb, None, None if klen is None else [klen], seed=77, fused=False)
    p.forward()
    grads = p.grads()
    p.backward(grads)
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    n = nk if klen is None else klen
    ref = p.reference()
    i = torch.arange(nq, device="cuda")[:, None] + nk - nq
    j = torch.arange(n, device="cuda")[None]
    see = torch.ones(nq, n, dtype=torch.bool, device="cuda")
    if cb:
        see = (i >= 0) & (torch.div(i, cb, rounding_mode="floor") >= torch.div(j, cb, rounding_mode="floor"))
    for h in range(H):
        at = slice(h * hd, (h + 1) * hd)
        q, k, v, do = (t.double() for t in (p.q[0, :, at], p.k[0, :n, at], p.v[0, :n, at], p.do[0, :, at]))
        pr = torch.nan_to_num(torch.softmax((q @ k.T / math.sqrt(hd)).masked_fill(~see, -math.inf), 1))
        dp, m = do @ v.T, do.abs() @ v.abs().T
        ds = pr * (dp - (pr * dp).sum(1, keepdim=True))
        ds_b = (U + F) * ds.abs() + pr * (F + 2.0 ** -20) * (m + (pr * m).sum(1, keepdim=True))
        for name, got, b in (("dq", grads[0][0, :, at], ds_b @ k.abs()), ("dk", grads[1][0, :n, at], ds_b.T @ q.abs())):
            want = ref[name][0, :got.shape[0], h]
            within(got, want, b / math.sqrt(hd) + U * want.abs() + 1e-30, name)
