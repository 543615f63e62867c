"""Cases of the training operators: attention with its row statistics and its
backward pass, LayerNorm and RMSNorm with theirs.

`run` computes one pass either in plain torch (float32, rounded once at the
end) or, where `own` is true, through the package's dlo_op_* calls.  Sizes are
those of the block stacks in synth/ (4 x 64, 16 x 72 and 40 x 128 heads, 256,
1024, 8192 and 32760 tokens, 512 text tokens) and generic odd ones.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _attn(name, op, batch, heads, kv_heads, head_dim, nq, nk, causal_block, lens):
    return {"name": name, "op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "nq": nq, "nk": nk, "causal_block": causal_block, "lens": lens}


def _ln(name, op, batch, tokens, dim, form):
    return {"name": name, "op": op, "batch": batch, "tokens": tokens, "dim": dim, "form": form}


def _rms(name, op, tokens, dim):
    return {"name": name, "op": op, "tokens": tokens, "dim": dim}


def listed():
    return [
        # the tiny stack's self-attention: one launch's latency
        _attn("attn fwd tiny", "attn_fwd", 1, 4, 4, 64, 256, 256, 0, "full"),
        # frame-causal video self-attention, 520 tokens a frame, videos of two lengths in a batch
        _attn("attn fwd frame-causal", "attn_fwd", 2, 24, 24, 128, 4680, 4680, 520, "ragged"),
        # few learned queries that read a long sequence through shared key/value heads
        _attn("attn fwd few queries", "attn_fwd", 2, 16, 4, 64, 37, 8192, 0, "full"),
        # DiT-XL self-attention's gradients
        _attn("attn bwd dit-xl", "attn_bwd", 2, 16, 16, 72, 1024, 1024, 0, "full"),
        # the video stack's self-attention at 8192 tokens: the largest
        _attn("attn bwd video", "attn_bwd", 1, 40, 40, 128, 8192, 8192, 0, "full"),
        # its cross-attention to 512 text tokens, prompts of several lengths
        _attn("attn bwd cross", "attn_bwd", 2, 40, 40, 128, 4095, 512, 0, "ragged"),
        # shared key/value heads, token-causal, an odd ragged batch with an empty sequence
        _attn("attn bwd causal shared", "attn_bwd", 3, 16, 4, 64, 2047, 2047, 1, "empty"),
        # DiT-XL adaLN
        _ln("layernorm fwd dit-xl", "ln_fwd", 2, 1024, 1152, "mod"),
        _ln("layernorm bwd dit-xl", "ln_bwd", 2, 1024, 1152, "mod"),
        # the video stack's affine LayerNorm before cross-attention, with its weight's gradient
        _ln("layernorm bwd video", "ln_bwd", 1, 32760, 5120, "affine"),
        # q/k norm of the video stack inside the fused q|k|v rows
        _rms("rmsnorm fwd video", "rms_fwd", 8192, 5120),
        _rms("rmsnorm bwd video", "rms_bwd", 8192, 5120),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "ln_fwd", "ln_bwd", "rms_fwd", "rms_bwd"])
    if op.startswith("attn"):
        while True:
            batch = rng.randint(1, 4)
            heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 40])
            kv = heads // rng.choice([g for g in (1, 1, 2, 3, 4, 8) if heads % g == 0])
            hd = rng.choice([16, 32, 40, 64, 64, 72, 80, 88, 96, 112, 128, 128])
            kind = rng.choice(["self", "self", "cross", "few"])
            n = _log_int(rng, 16, 8192)
            if kind == "self":
                nq = nk = n
            elif kind == "cross":
                nq, nk = n, _log_int(rng, 16, 600)
            else:
                nq, nk = _log_int(rng, 1, 128), n
            if batch * heads * nq * nk * hd <= 40 * 8192 * 8192 * 128 // 2:
                break
        block = rng.choice([0, 0, 1, _log_int(rng, 2, 700)])
        lens = rng.choice(["full", "ragged", "empty"]) if batch > 1 else "full"
        return _attn("", op, batch, heads, kv, hd, nq, nk, block, lens) | {"name": "%s %dx%d/%dx%d %dx%d" % (
            op, batch, heads, kv, hd, nq, nk)}
    if op.startswith("ln"):
        while True:
            batch, tokens, dim = rng.randint(1, 4), _log_int(rng, 1, 32760), 4 * _log_int(rng, 16, 2048)
            if batch * tokens * dim <= 32760 * 5120:
                break
        form = rng.choice(["mod", "affine", "plain"])
        return _ln("%s %s %dx%dx%d" % (op, form, batch, tokens, dim), op, batch, tokens, dim, form)
    while True:
        tokens, dim = _log_int(rng, 1, 32760), 8 * _log_int(rng, 8, 1024)
        if tokens * dim <= 32760 * 5120 // 2:
            break
    return _rms("%s %dx%d" % (op, tokens, dim), op, tokens, dim)


# ------------------------------------------------------------------ inputs

def _lens(case, n):
    """Valid tokens of each sequence of the batch (None: all of them)."""
    b = case["batch"]
    if case["lens"] == "full":
        return None
    lens = [n - (i * n * 5) // (8 * b) for i in range(b)]
    if case["lens"] == "empty":
        lens[-1] = 0
    return lens


def _int32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _split(case, qkv):
    """q, k and v as views of the fused rows q | k | v (one buffer, the block's own layout) or of q and k | v."""
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    if len(qkv) == 1:
        return qkv[0].split([h * d, g * d, g * d], dim=-1)
    return (qkv[0],) + tuple(qkv[1].split([g * d, g * d], dim=-1))


def _attn_rows(case, make):
    b, h, g, d, nq, nk = (case[k] for k in ("batch", "heads", "kv_heads", "head_dim", "nq", "nk"))
    if nq == nk:
        return [make((b, nq, (h + 2 * g) * d))]
    return [make((b, nq, h * d)), make((b, nk, 2 * g * d))]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def empty(shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=DEV)

    if op.startswith("attn"):
        b, h, d, nq = case["batch"], case["heads"], case["head_dim"], case["nq"]
        # q and k come out of RMSNorm: unit variance, logits of order one
        s["qkv"] = _attn_rows(case, lambda shape: _normal(gen, shape))
        s["q"], s["k"], s["v"] = _split(case, s["qkv"])
        s["q_lens"] = _int32(_lens(case, nq))
        s["k_lens"] = _int32(_lens(case, case["nk"]))
        if op == "attn_bwd":
            # what the forward pass left, and the gradient that arrives from the projection behind it
            s["o"], s["lse"] = _attn_fwd_plain(s)
            s["do"] = _normal(gen, (b, nq, h * d), 0.02)
        if own:
            _attn_plan(s, empty)
    elif op.startswith("ln"):
        b, n, d = case["batch"], case["tokens"], case["dim"]
        # a residual stream: rows of different scale, with an offset
        s["x"] = _normal(gen, (b, n, d), 1.0, torch.float32) * (0.5 + torch.rand((b, n, 1), generator=gen, device=DEV) * 2) + 0.1
        if case["form"] == "mod":
            s["mod"] = _normal(gen, (b, 6 * d), 0.3, torch.float32)
        elif case["form"] == "affine":
            s["w"] = _normal(gen, (d,), 0.02) + 1
            s["b"] = _normal(gen, (d,), 0.02)
        if op == "ln_bwd":
            s["mean"], s["rstd"] = _ln_stats(s["x"])
            s["dy"] = _normal(gen, (b, n, d), 0.02)
            s["dres"] = _normal(gen, (b, n, d), 0.02, torch.float32)
        if own:
            _ln_plan(s, empty)
    else:
        n, d = case["tokens"], case["dim"]
        s["qkv"] = _normal(gen, (n, 3 * d))       # k of fused q | k | v rows
        s["w"] = _normal(gen, (d,), 0.02) + 1
        if op == "rms_bwd":
            x = s["qkv"][:, d:2 * d].float()
            s["rstd"] = torch.rsqrt((x * x).mean(-1) + EPS)
            s["dy"] = _normal(gen, (n, 3 * d), 0.02)
        if own:
            _rms_plan(s, empty)
    return s


# ------------------------------------------------------------------ plain forms

def _visible(s):
    """[batch, 1, nq, nk] truth values of which query sees which key."""
    c = s["case"]
    i = torch.arange(c["nq"], device=DEV)[:, None] + (c["nk"] - c["nq"])
    j = torch.arange(c["nk"], device=DEV)[None, :]
    see = torch.ones((1, c["nq"], c["nk"]), dtype=torch.bool, device=DEV)
    if c["causal_block"]:
        n = c["causal_block"]
        see = see & (i >= 0) & (torch.div(i, n, rounding_mode="floor") >= torch.div(j, n, rounding_mode="floor"))
    if s["q_lens"] is not None:
        see = see & (torch.arange(c["nq"], device=DEV)[None, :, None] < s["q_lens"][:, None, None])
        see = see & (j[None] < s["k_lens"][:, None, None])
    return see[:, None]


def _heads(s, x, n):
    """[batch, rows, n * hd] -> float32 [batch, heads, rows, hd], shared heads repeated."""
    c = s["case"]
    x = x.float().reshape(x.shape[0], x.shape[1], n, c["head_dim"]).transpose(1, 2)
    return x.repeat_interleave(c["heads"] // n, dim=1)


def _rows(x):
    return x.transpose(1, 2).reshape(x.shape[0], x.shape[2], -1)


def _probabilities(s):
    c = s["case"]
    q = _heads(s, s["q"], c["heads"])
    k = _heads(s, s["k"], c["kv_heads"])
    see = _visible(s)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(c["head_dim"])).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)          # log 0 = -inf where nothing is visible
    return q, k, x.div_(torch.where(total == 0, torch.ones_like(total), total)), lse


def _attn_fwd_plain(s):
    c = s["case"]
    _, _, p, lse = _probabilities(s)
    v = _heads(s, s["v"], c["kv_heads"])
    return _rows(torch.matmul(p, v)).to(torch.bfloat16), lse


def _shared(s, x):
    c = s["case"]
    g = c["kv_heads"]
    return x.reshape(x.shape[0], g, c["heads"] // g, x.shape[2], x.shape[3]).sum(2)


def _attn_bwd_plain(s):
    c = s["case"]
    q, k, p, _ = _probabilities(s)
    v = _heads(s, s["v"], c["kv_heads"])
    do = _heads(s, s["do"], c["heads"])
    dv = torch.matmul(p.transpose(-1, -2), do)
    dp = torch.matmul(do, v.transpose(-1, -2))
    dp = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(c["head_dim"]))
    dq = torch.matmul(dp, k)
    dk = torch.matmul(dp.transpose(-1, -2), q)
    return [_rows(x).to(torch.bfloat16) for x in (dq, _shared(s, dk), _shared(s, dv))]


def _ln_stats(x):
    mean = x.mean(-1)
    var = (x - mean[..., None]).square().mean(-1)
    return mean, torch.rsqrt(var + EPS)


def _ln_gain(s):
    """What multiplies the normalised row, and what is added to it (0-dim ones where there is nothing)."""
    if s["case"]["form"] == "mod":
        d = s["case"]["dim"]
        return 1 + s["mod"][:, None, d:2 * d], s["mod"][:, None, :d]
    if s["case"]["form"] == "affine":
        return s["w"].float(), s["b"].float()
    return torch.ones((), device=DEV), torch.zeros((), device=DEV)


def _ln_fwd_plain(s):
    mean, rstd = _ln_stats(s["x"])
    gain, shift = _ln_gain(s)
    xh = (s["x"] - mean[..., None]) * rstd[..., None]
    return [(xh * gain + shift).to(torch.bfloat16), mean, rstd]


def _ln_bwd_plain(s):
    xh = (s["x"] - s["mean"][..., None]) * s["rstd"][..., None]
    gain, _ = _ln_gain(s)
    dy = s["dy"].float()
    g = dy * gain
    dx = s["rstd"][..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True)) + s["dres"]
    if s["case"]["form"] == "plain":
        return [dx]
    over = 1 if s["case"]["form"] == "mod" else (0, 1)
    return [dx, dy.sum(over), (dy * xh).sum(over)]


def _rms_fwd_plain(s):
    d = s["case"]["dim"]
    x = s["qkv"][:, d:2 * d].float()
    r = torch.rsqrt((x * x).mean(-1) + EPS)
    return [(x * r[:, None] * s["w"].float()).to(torch.bfloat16), r]


def _rms_bwd_plain(s):
    d = s["case"]["dim"]
    x, dy = s["qkv"][:, d:2 * d].float(), s["dy"][:, d:2 * d].float()
    xh = x * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    return [dx.to(torch.bfloat16), (dy * xh).sum(0)]


# ------------------------------------------------------------------ the package's calls

def _dlo():
    import layerwise_weight_offload_slot_gb300 as dlo
    return dlo


def _workspace(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _attn_plan(s, empty):
    """The call's description, output buffers and workspace, as a training program keeps them."""
    dlo, c = _dlo(), s["case"]
    b, h, d, nq = c["batch"], c["heads"], c["head_dim"], c["nq"]
    ld = {"ldq": s["q"].stride(1), "ldk": s["k"].stride(1), "ldv": s["v"].stride(1), "ldo": h * d}
    if c["op"] == "attn_bwd":
        s["dqkv"] = _attn_rows(c, empty)
        s["dq"], s["dk"], s["dv"] = _split(c, s["dqkv"])
        ld |= {"lddq": s["dq"].stride(1), "lddk": s["dk"].stride(1), "lddv": s["dv"].stride(1), "lddo": h * d}
    else:
        s["o"], s["lse"] = empty((b, nq, h * d)), empty((b, h, nq), torch.float32)
    a = dlo.make_attn(batch=b, heads=h, kv_heads=c["kv_heads"], head_dim=d, nq=nq, nk=c["nk"],
                      causal_block=c["causal_block"], q_lens=_ptr(s["q_lens"]), k_lens=_ptr(s["k_lens"]), **ld)
    size = dlo.dlo_attention_bwd_workspace_bytes if c["op"] == "attn_bwd" else dlo.dlo_attention_fwd_workspace_bytes
    s["attn"], s["ws"] = a, _workspace(size(a))
    s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)


def _ln_plan(s, empty):
    dlo, c = _dlo(), s["case"]
    b, n, d = c["batch"], c["tokens"], c["dim"]
    if c["op"] == "ln_fwd":
        s["y"], s["mean"], s["rstd"] = empty((b, n, d)), empty((b, n), torch.float32), empty((b, n), torch.float32)
        return
    s["dx"] = empty((b, n, d), torch.float32)
    if c["form"] == "mod":
        s["dmod"] = torch.zeros((b, 6 * d), dtype=torch.float32, device=DEV)
    elif c["form"] == "affine":
        s["dw"], s["db"] = empty((d,), torch.float32), empty((d,), torch.float32)
    s["ws"] = _workspace(dlo.dlo_layernorm_bwd_workspace_bytes(b * n, d, n))


def _rms_plan(s, empty):
    dlo, c = _dlo(), s["case"]
    n, d = c["tokens"], c["dim"]
    if c["op"] == "rms_fwd":
        s["y"], s["rstd"] = empty((n, d)), empty((n,), torch.float32)
        return
    s["dx"], s["dw"] = empty((n, 3 * d)), empty((d,), torch.float32)
    s["ws"] = _workspace(dlo.dlo_rmsnorm_bwd_workspace_bytes(n, d))


def _run_own(s):
    dlo, c, op = _dlo(), s["case"], s["case"]["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "attn_fwd":
        dlo.dlo_op_attention_fwd(s["attn"], s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(),
                                 s["o"].data_ptr(), s["lse"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(),
                                 s["err"].data_ptr(), stream)
        return [s["o"], s["lse"]]
    if op == "attn_bwd":
        dlo.dlo_op_attention_bwd(s["attn"], s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(),
                                 s["o"].data_ptr(), s["lse"].data_ptr(), s["do"].data_ptr(), s["dq"].data_ptr(),
                                 s["dk"].data_ptr(), s["dv"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(),
                                 s["err"].data_ptr(), stream)
        return [s["dq"], s["dk"], s["dv"]]
    if op.startswith("ln"):
        b, n, d, form = c["batch"], c["tokens"], c["dim"], c["form"]
        shift = s["mod"][:, :d].data_ptr() if form == "mod" else None
        scale = s["mod"][:, d:].data_ptr() if form == "mod" else None
        w = _ptr(s.get("w"))
        if op == "ln_fwd":
            dlo.dlo_op_layernorm_fwd(s["x"].data_ptr(), b * n, d, n, shift, scale, 6 * d, w, _ptr(s.get("b")), EPS,
                                     s["y"].data_ptr(), s["mean"].data_ptr(), s["rstd"].data_ptr(), stream)
            return [s["y"], s["mean"], s["rstd"]]
        dshift = s["dmod"][:, :d] if form == "mod" else s.get("db")
        dscale = s["dmod"][:, d:2 * d] if form == "mod" else s.get("dw")
        dlo.dlo_op_layernorm_bwd(s["dy"].data_ptr(), s["x"].data_ptr(), s["mean"].data_ptr(), s["rstd"].data_ptr(),
                                 b * n, d, n, scale, 6 * d, w, s["dres"].data_ptr(), s["dx"].data_ptr(),
                                 _ptr(dshift), _ptr(dscale), 6 * d, s["ws"].data_ptr(), s["ws"].numel(), stream)
        return [s["dx"]] if form == "plain" else [s["dx"], dshift, dscale]
    n, d = c["tokens"], c["dim"]
    x = s["qkv"][:, d:]
    if op == "rms_fwd":
        dlo.dlo_op_rmsnorm_fwd(x.data_ptr(), 3 * d, n, d, s["w"].data_ptr(), EPS, s["y"].data_ptr(), d,
                               s["rstd"].data_ptr(), stream)
        return [s["y"], s["rstd"]]
    dx = s["dx"][:, d:2 * d]
    dlo.dlo_op_rmsnorm_bwd(s["dy"][:, d:].data_ptr(), 3 * d, x.data_ptr(), 3 * d, s["w"].data_ptr(),
                           s["rstd"].data_ptr(), n, d, dx.data_ptr(), 3 * d, s["dw"].data_ptr(),
                           s["ws"].data_ptr(), s["ws"].numel(), stream)
    return [dx, s["dw"]]


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "attn_fwd":
        return list(_attn_fwd_plain(s))
    return {"attn_bwd": _attn_bwd_plain, "ln_fwd": _ln_fwd_plain, "ln_bwd": _ln_bwd_plain,
            "rms_fwd": _rms_fwd_plain, "rms_bwd": _rms_bwd_plain}[op](s)


# ------------------------------------------------------------------ work

def _pairs(case):
    """Visible (query, key) pairs of one head, over the batch."""
    nq, nk, n = case["nq"], case["nk"], case["causal_block"]
    ql, kl = _lens(case, nq) or [nq] * case["batch"], _lens(case, nk) or [nk] * case["batch"]
    total = 0
    for a, b in zip(ql, kl):
        if not n:
            total += a * b
        else:
            total += sum(min(b, ((i + nk - nq) // n + 1) * n) for i in range(max(0, nq - nk), a))
    return total


def work(case):
    op = case["op"]
    if op.startswith("attn"):
        h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
        rq = sum(_lens(case, case["nq"]) or [case["nq"]] * case["batch"])
        rk = sum(_lens(case, case["nk"]) or [case["nk"]] * case["batch"])
        q, kv, lse = 2 * rq * h * d, 2 * rk * g * d, 4 * rq * h
        pairs = _pairs(case) * h * d
        if op == "attn_fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * pairs}
    if op.startswith("ln"):
        rows, d = case["batch"] * case["tokens"], case["dim"]
        par = {"mod": 8 * case["batch"] * d, "affine": 4 * d, "plain": 0}[case["form"]]
        if op == "ln_fwd":
            return {"bytes": rows * (6 * d + 8) + par, "flops": 8 * rows * d}
        gain = {"mod": 12 * case["batch"] * d, "affine": 10 * d, "plain": 0}[case["form"]]
        return {"bytes": rows * (14 * d + 8) + gain, "flops": 14 * rows * d}
    rows, d = case["tokens"], case["dim"]
    if op == "rms_fwd":
        return {"bytes": rows * (4 * d + 4) + 2 * d, "flops": 4 * rows * d}
    return {"bytes": rows * (6 * d + 4) + 6 * d, "flops": 10 * rows * d}


# ------------------------------------------------------------------ in 64 bits

def _exact_attention(s):
    """The definition, one (sequence, head) at a time over its valid rows only; gradients where there is a `do`."""
    c = s["case"]
    b, h, g, d, nq, nk = (c[k] for k in ("batch", "heads", "kv_heads", "head_dim", "nq", "nk"))
    f64 = {"dtype": torch.float64, "device": DEV}
    o, lse = torch.zeros((b, nq, h, d), **f64), torch.full((b, h, nq), -math.inf, **f64)
    dq, dk, dv = torch.zeros((b, nq, h, d), **f64), torch.zeros((b, nk, g, d), **f64), torch.zeros((b, nk, g, d), **f64)
    q, k, v = s["q"].view(b, nq, h, d), s["k"].view(b, nk, g, d), s["v"].view(b, nk, g, d)
    ql, kl = _lens(c, nq) or [nq] * b, _lens(c, nk) or [nk] * b
    for n in range(b):
        first = max(0, nq - nk) if c["causal_block"] else 0
        if ql[n] <= first or kl[n] == 0:
            continue
        rows = torch.arange(first, ql[n], device=DEV)
        last = torch.full_like(rows, kl[n])           # one past the last key that a row sees
        if c["causal_block"]:
            last = torch.minimum(last, ((rows + (nk - nq)) // c["causal_block"] + 1) * c["causal_block"])
        hidden = torch.arange(kl[n], device=DEV)[None, :] >= last[:, None]
        for m in range(h):
            e = m * g // h
            qq, kk, vv = q[n, first:ql[n], m].double(), k[n, :kl[n], e].double(), v[n, :kl[n], e].double()
            x = (qq @ kk.T) / math.sqrt(d)
            x[hidden] = -math.inf
            lse[n, m, first:ql[n]] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[n, m, first:ql[n], None])
            o[n, first:ql[n], m] = p @ vv
            if "do" in s:
                do = s["do"].view(b, nq, h, d)[n, first:ql[n], m].double()
                dv[n, :kl[n], e] += p.T @ do
                ds = p * (do @ vv.T - (do * o[n, first:ql[n], m]).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[n, first:ql[n], m] = ds @ kk
                dk[n, :kl[n], e] += ds.T @ qq
    if "do" in s:
        return [dq.flatten(2), dk.flatten(2), dv.flatten(2)]
    return [o.flatten(2), lse]


def _exact_layernorm(s):
    c, x = s["case"], s["x"].double()
    d = c["dim"]
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    std = torch.sqrt(var + EPS)
    gain = {"mod": lambda: 1 + s["mod"][:, d:2 * d].double().unsqueeze(1), "affine": lambda: s["w"].double(), "plain": lambda: 1.0}[c["form"]]()
    if c["op"] == "ln_fwd":
        add = {"mod": lambda: s["mod"][:, :d].double().unsqueeze(1), "affine": lambda: s["b"].double(), "plain": lambda: 0.0}[c["form"]]()
        return [(x - mean) / std * gain + add, mean.squeeze(-1), 1 / std.squeeze(-1)]
    dy = s["dy"].double()
    xh = (x - mean) / std
    g = dy * gain
    dx = (d * g - g.sum(-1, keepdim=True) - xh * (g * xh).sum(-1, keepdim=True)) / (d * std) + s["dres"].double()
    if c["form"] == "plain":
        return [dx]
    both = [dy, dy * xh]
    if c["form"] == "affine":
        both = [t.flatten(0, 1).unsqueeze(0) for t in both]
    both = [t.sum(1) for t in both]
    return [dx] + ([t[0] for t in both] if c["form"] == "affine" else both)


def _exact_rmsnorm(s):
    d = s["case"]["dim"]
    x = s["qkv"][:, d:2 * d].double()
    rms = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + EPS)
    w = s["w"].double()
    if s["case"]["op"] == "rms_fwd":
        return [x / rms * w, 1 / rms.squeeze(-1)]
    dy = s["dy"][:, d:2 * d].double()
    dot = (dy * w * x).sum(-1, keepdim=True)
    return [dy * w / rms - x * dot / (d * rms.pow(3)), torch.einsum("nd,nd->d", dy, x / rms)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attention(s)
    return _exact_layernorm(s) if case["op"].startswith("ln") else _exact_rmsnorm(s)
