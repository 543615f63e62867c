"""Cases of the operators for packed batches: the plan of a packed batch (row starts and positions), rotary
positions, and attention over packed sequences, each with its gradient where it has one.

`run` computes one pass either in plain torch (float32, angles in 64 bits, rounded once at the end) or, where `own`
is true, through the package's calls.  Sizes are those of the block stacks in synth/ (4 x 64, 16 x 72 and 40 x 128
heads, 1024 and 8192 tokens, 512 text tokens, frames of 520) and generic odd ones.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
#
# Sequences of a packed batch are given by `batch`, `rows` (their sum) and how the lengths differ:
#   even    alike up to one row            mixed   from about a tenth of the mean to twice the mean
#   long    one sequence has half of all rows
#   empty   as mixed, and every fifth sequence has no rows
# `slack` rows of each buffer lie behind the last sequence.

def _plan(name, batch, rows, axes, lens, slack):
    return {"name": name, "op": "plan", "batch": batch, "rows": rows, "axes": axes, "lens": lens, "slack": slack}


def _rope(name, op, rows, heads, behind, head_dim, rot, axes, layout, scaling, far):
    """`heads` of the fused rows are rotated, `behind` more (the values) follow them; positions from `far` on."""
    return {"name": name, "op": op, "rows": rows, "heads": heads, "behind": behind, "head_dim": head_dim, "rot": rot,
            "axes": axes, "layout": layout, "scaling": scaling, "far": far}


def _attn(name, op, batch, heads, kv_heads, head_dim, rows, keys, causal_block, lens, slack):
    """`keys` 0: self-attention over the same rows; else `keys` rows of keys of the same sequences, packed apart."""
    return {"name": name, "op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rows": rows, "keys": keys, "causal_block": causal_block, "lens": lens, "slack": slack}


def listed():
    return [
        # a few images of a small batch: one launch's latency
        _plan("plan images", 6, 1500, 2, "mixed", 36),
        # many clips, (frame, row, column) of every token
        _plan("plan clips", 300, 32760, 3, "mixed", 8),
        # the next token of each of a few sequences, far into a context that was scaled eightfold
        _rope("rope fwd single tokens", "rope_fwd", 24, 20, 4, 128, 128, 1, "half", "turns", 100000),
        # q and k of the video stack inside fused q | k | v rows, (frame, row, column)
        _rope("rope fwd video", "rope_fwd", 8192, 80, 40, 128, 128, 3, "interleaved", "none", 0),
        # their gradients on the way back, long prompts, a part of each head
        _rope("rope bwd part", "rope_bwd", 16381, 48, 16, 96, 72, 1, "half", "index", 0),
        # the tiny stack's self-attention over three small images
        _attn("packed fwd tiny", "attn_fwd", 3, 4, 4, 64, 256, 0, 0, "mixed", 0),
        # DiT-XL self-attention over images of many resolutions
        _attn("packed fwd images", "attn_fwd", 24, 16, 16, 72, 8190, 0, 0, "mixed", 2),
        # prompts of different lengths, token-causal, shared key/value heads
        _attn("packed fwd prompts", "attn_fwd", 9, 40, 8, 128, 16381, 0, 1, "empty", 3),
        # one query for each sequence against its cached keys and values
        _attn("packed fwd single queries", "attn_fwd", 24, 40, 8, 128, 24, 98304, 1, "mixed", 0),
        # DiT-XL training on the images
        _attn("packed bwd images", "attn_bwd", 24, 16, 16, 72, 8190, 0, 0, "mixed", 2),
        # the video stack, frame-causal clips, one of them much longer: the largest
        _attn("packed bwd clips", "attn_bwd", 5, 40, 40, 128, 12480, 0, 520, "long", 0),
        # its cross-attention to the text tokens of each clip
        _attn("packed bwd text", "attn_bwd", 6, 40, 40, 128, 8189, 1700, 0, "mixed", 3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope_fwd", "rope_bwd", "attn_fwd", "attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd"])
    lens = rng.choice(["even", "mixed", "mixed", "long", "empty"])
    slack = rng.choice([0, 0, 1, 7, 130])
    if op == "plan":
        batch, axes = _log_int(rng, 1, 600), rng.choice([1, 2, 3])
        rows = _log_int(rng, max(16, batch), 32760)
        return _plan("plan %dx%d/%d" % (batch, axes, rows), batch, rows, axes, lens, slack)
    if op.startswith("rope"):
        while True:
            rows, heads = _log_int(rng, 1, 32760), rng.choice([1, 3, 4, 8, 20, 32, 48, 80])
            hd = rng.choice([32, 40, 64, 72, 80, 96, 128, 128])
            if rows * heads * hd <= 8192 * 80 * 128:
                break
        axes = rng.choice([1, 1, 2, 3])
        rot = rng.choice([hd, hd, hd, hd // 2, hd * 3 // 4 // 4 * 4, 20])
        return _rope("%s %dx%dx%d/%d" % (op, rows, heads, hd, rot), op, rows, heads, rng.choice([0, 0, heads]), hd, rot, axes,
                     rng.choice(["interleaved", "half"]), rng.choice(["none", "linear", "base", "turns", "index"]),
                     rng.choice([0, 0, 1000, 200000]))
    while True:
        batch = _log_int(rng, 1, 64)
        heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 40])
        kv = heads // rng.choice([g for g in (1, 1, 2, 3, 4, 5, 8) if heads % g == 0])
        hd = rng.choice([16, 32, 40, 64, 64, 72, 80, 88, 96, 112, 128, 128])
        kind = rng.choice(["self", "self", "self", "cross", "few", "single"])
        rows, keys = _log_int(rng, max(32, 2 * batch), 16384), 0
        if kind == "cross":
            keys = _log_int(rng, batch, 2048)
        elif kind == "few":
            rows, keys = _log_int(rng, batch, 16 * batch), _log_int(rng, 4 * batch, 65536)
        elif kind == "single":
            op, rows, keys = "attn_fwd", batch, _log_int(rng, 16 * batch, 98304)
        block = rng.choice([0, 0, 1, 1, _log_int(rng, 2, 700)])
        c = _attn("%s %s %dx%d/%dx%d %dx%d" % (op, kind, batch, heads, kv, hd, rows, keys), op, batch, heads, kv, hd, rows, keys,
                  block, lens, slack)
        # no dearer than the largest listed cases
        if work(c)["flops"] <= 1.4e12 and (keys or rows) * kv * hd <= 98304 * 8 * 128:
            return c


def _lengths(batch, total, how):
    """`batch` lengths that add up to `total`."""
    if how == "even":
        weight = [1] * batch
    elif how == "long":
        weight = [1] * batch
        weight[batch // 2] = max(1, batch - 1)
    else:
        weight = [2 + (7 * i + 5) % 19 * 2 for i in range(batch)]
        if how == "empty":
            weight = [0 if i % 5 == 3 else w for i, w in enumerate(weight)]
    whole = sum(weight)
    ends = [total * sum(weight[:i + 1]) // whole for i in range(batch)]
    return [e - s for s, e in zip([0] + ends, ends)]


def _q_lengths(case):
    if case["keys"] and case["rows"] == case["batch"]:
        return [1] * case["batch"]
    return _lengths(case["batch"], case["rows"], case["lens"])


def _k_lengths(case):
    return _lengths(case["batch"], case["keys"], case["lens"]) if case["keys"] else _q_lengths(case)


def _grids(case):
    """Extents of each sequence, whose products are about the lengths and together at most `rows`."""
    out = []
    for n in _lengths(case["batch"], case["rows"], case["lens"]):
        if case["axes"] == 1:
            out.append([n])
        elif case["axes"] == 2:
            w = max(1, math.isqrt(n))
            out.append([n // w, w])
        else:
            w = max(1, round(n ** (1 / 3)))
            out.append([n // (w * w), w, w])
    return out


def _axes(case):
    """[(columns, base, scaling, factor)] of each rotary axis: the columns are split in even parts, the first gets the rest."""
    n, rot = case["axes"], case["rot"]
    part = rot // n // 2 * 2
    dims = [rot - (n - 1) * part] + [part] * (n - 1)
    return [(d, 10000.0, case["scaling"], 8.0) for d in dims]


# what the blended scalings go by: the context that was trained on, and between how many turns in it they blend
LENGTH, FAST, SLOW = 8192.0, 32.0, 1.0


# ------------------------------------------------------------------ inputs

def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _zeros(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _split(case, qkv):
    """q, k and v as views of the fused rows q | k | v, or of q and k | v."""
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    if len(qkv) == 1:
        return qkv[0].split([h * d, g * d, g * d], dim=-1)
    return (qkv[0],) + tuple(qkv[1].split([g * d, g * d], dim=-1))


def _attn_rows(case, make):
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    rows, keys = case["rows"] + case["slack"], case["keys"] + case["slack"]
    if not case["keys"]:
        return [make((rows, (h + 2 * g) * d))]
    return [make((rows, h * d)), make((keys, 2 * g * d))]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "plan":
        grids = _grids(case)
        # another seed brings the same sequences in another order, and other places to go on from
        order = torch.randperm(len(grids), generator=gen, device=DEV).tolist()
        s["host_grids"] = [grids[i] for i in order]
        s["grids"] = _int32(s["host_grids"])
        s["offsets"] = torch.randint(0, 5000, (len(grids), case["axes"]), generator=gen, device=DEV, dtype=torch.int32)
        if own:
            s["starts"] = _zeros((len(grids) + 1,), torch.int32)
            s["positions"] = _zeros((case["rows"] + case["slack"], case["axes"]), torch.int32)
    elif op.startswith("rope"):
        n, hd = case["rows"], case["head_dim"]
        wide, narrow = (case["heads"] + case["behind"]) * hd, case["heads"] * hd
        # forward: q and k inside fused rows to rows of their own; backward: the other way round
        s["x"] = _normal(gen, (n, wide)) if op == "rope_fwd" else _normal(gen, (n, narrow), 0.02)
        at = case["far"] + torch.randint(0, max(1, n), (n, case["axes"]), generator=gen, device=DEV, dtype=torch.int32)
        s["positions"] = at.contiguous()
        if own:
            _rope_plan(s)
    else:
        s["qkv"] = _attn_rows(case, lambda shape: _normal(gen, shape))
        s["q"], s["k"], s["v"] = _split(case, s["qkv"])
        s["q_starts"] = _int32(_starts(_q_lengths(case)))
        s["k_starts"] = _int32(_starts(_k_lengths(case))) if case["keys"] else s["q_starts"]
        if op == "attn_bwd":
            # what the forward pass left, and the gradient that arrives from the projection behind it
            s["o"], s["lse"] = _attn_fwd_plain(s)
            s["do"] = _normal(gen, s["o"].shape, 0.02)
        if own:
            _attn_plan(s)
    return s


# ------------------------------------------------------------------ plain forms

def _plan_plain(s):
    c = s["case"]
    grids = s["grids"].long()
    lens = grids.prod(1)
    starts = torch.zeros(c["batch"] + 1, dtype=torch.int64, device=DEV)
    starts[1:] = lens.cumsum(0)
    positions = _zeros((c["rows"] + c["slack"], c["axes"]), torch.int32)
    seq = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), lens)
    i = torch.arange(seq.numel(), device=DEV) - starts[seq]
    for a in reversed(range(c["axes"])):
        n = grids[seq, a]
        positions[:seq.numel(), a] = (i % n + s["offsets"][seq, a]).int()
        i = torch.div(i, n, rounding_mode="floor")
    return [starts.int(), positions]


def _frequencies(case):
    """Radians a position of every pair, in 64 bits, and the axis that it follows."""
    out, axis = [], []
    for a, (dim, base, scaling, factor) in enumerate(_axes(case)):
        p = torch.arange(dim // 2, dtype=torch.float64, device=DEV)
        if scaling == "base" and dim > 2:
            base = base * factor ** (dim / (dim - 2))
        f = base ** (-2 * p / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "turns":
            keep = ((LENGTH * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
            f = f * (keep + (1 - keep) / factor)
        elif scaling == "index":
            at = [dim * math.log(LENGTH / (2 * math.pi * t)) / (2 * math.log(base)) for t in (FAST, SLOW)]
            low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
            keep = 1 - ((p - low) / max(high - low, 0.001)).clamp(0, 1)
            f = f * (keep + (1 - keep) / factor)
        out.append(f)
        axis += [a] * (dim // 2)
    return torch.cat(out), axis


AMP = 1.125


def _rope_plain(s):
    c = s["case"]
    n, h, hd, rot = c["rows"], c["heads"], c["head_dim"], c["rot"]
    f, axis = _frequencies(c)
    angle = s["positions"].double()[:, axis] * f
    cos, sin = (AMP * angle.cos()).float()[:, None], (AMP * angle.sin()).float()[:, None]
    if c["op"] == "rope_bwd":
        sin = -sin
    x = s["x"][:, :h * hd].float().view(n, h, hd)
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y.view(n, h * hd).to(torch.bfloat16)


def _sequences(case):
    """(first query row, queries, first key row, keys) of every sequence."""
    ql, kl = _q_lengths(case), _k_lengths(case)
    return list(zip(_starts(ql), ql, _starts(kl), kl))


def _heads(case, x, n, first, rows):
    """Rows of one sequence -> float32 [heads, rows, hd], shared heads repeated."""
    x = x[first:first + rows].float().view(rows, n, case["head_dim"]).transpose(0, 1)
    return x.repeat_interleave(case["heads"] // n, dim=0)


def _probabilities(s, q0, nq, k0, nk):
    c = s["case"]
    q = _heads(c, s["q"], c["heads"], q0, nq)
    k = _heads(c, s["k"], c["kv_heads"], k0, nk)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(c["head_dim"]))
    if c["causal_block"]:
        i = torch.arange(nq, device=DEV)[:, None] + (nk - nq)
        j = torch.arange(nk, device=DEV)[None, :]
        block = c["causal_block"]
        see = (i >= 0) & (torch.div(i, block, rounding_mode="floor") >= torch.div(j, block, rounding_mode="floor"))
        x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)          # log 0 = -inf where nothing is visible
    return q, k, x.div_(torch.where(total == 0, torch.ones_like(total), total)), lse


def _put(out, first, x):
    """[heads, rows, hd] to the rows of one sequence."""
    out[first:first + x.shape[1]] = x.transpose(0, 1).reshape(x.shape[1], -1).to(out.dtype)


def _attn_fwd_plain(s):
    c = s["case"]
    rows = c["rows"] + c["slack"]
    o = _zeros((rows, c["heads"] * c["head_dim"]))
    lse = _zeros((c["heads"], rows), torch.float32)
    for q0, nq, k0, nk in _sequences(c):
        if nq and nk:
            _, _, p, l = _probabilities(s, q0, nq, k0, nk)
            _put(o, q0, torch.matmul(p, _heads(c, s["v"], c["kv_heads"], k0, nk)))
            lse[:, q0:q0 + nq] = l
        else:
            lse[:, q0:q0 + nq] = -math.inf
    return [o, lse]


def _attn_bwd_plain(s):
    c = s["case"]
    h, g, d = c["heads"], c["kv_heads"], c["head_dim"]
    grads = _attn_rows(c, _zeros)
    out_q, out_k, out_v = _split(c, grads)
    for q0, nq, k0, nk in _sequences(c):
        if not (nq and nk):
            continue
        q, k, p, _ = _probabilities(s, q0, nq, k0, nk)
        v = _heads(c, s["v"], g, k0, nk)
        do = _heads(c, s["do"], h, q0, nq)
        dv = torch.matmul(p.transpose(-1, -2), do)
        dp = torch.matmul(do, v.transpose(-1, -2))
        dp = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(d))
        _put(out_q, q0, torch.matmul(dp, k))
        _put(out_k, k0, torch.matmul(dp.transpose(-1, -2), q).view(g, h // g, nk, d).sum(1))
        _put(out_v, k0, dv.view(g, h // g, nk, d).sum(1))
    return [out_q, out_k, out_v]


# ------------------------------------------------------------------ the package's calls

def _dlo():
    import layerwise_weight_offload_slot_gb300 as dlo
    return dlo


def _rope_plan(s):
    """The call's description, its table of steps on the device and the rows it writes."""
    dlo, c = _dlo(), s["case"]
    hd = c["head_dim"]
    kinds = {"none": dlo.ROPE_PLAIN, "linear": dlo.ROPE_LINEAR, "base": dlo.ROPE_BASE, "turns": dlo.ROPE_BY_TURNS,
             "index": dlo.ROPE_BY_INDEX}
    axes = [dict(dim=d, theta=base, scaling=kinds[k], factor=factor, length=LENGTH, fast=FAST, slow=SLOW)
            for d, base, k, factor in _axes(c)]
    s["rope"] = dlo.make_rope(heads=c["heads"], head_dim=hd, axes=axes, amp=AMP, ldx=(c["heads"] + c["behind"]) * hd,
                              ldy=c["heads"] * hd,
                              layout=dlo.ROPE_HALF if c["layout"] == "half" else dlo.ROPE_INTERLEAVED)
    s["steps"] = torch.from_numpy(dlo.dlo_rope_steps(s["rope"])).to(DEV)
    wide = c["heads"] + (c["behind"] if c["op"] == "rope_bwd" else 0)
    s["y"] = _zeros((c["rows"], wide * hd))


def _attn_plan(s):
    """The call's description, output buffers and workspace, as a program keeps them."""
    dlo, c = _dlo(), s["case"]
    h, d = c["heads"], c["head_dim"]
    ld = {"ldq": s["q"].stride(0), "ldk": s["k"].stride(0), "ldv": s["v"].stride(0), "ldo": h * d}
    if c["op"] == "attn_bwd":
        s["grads"] = _attn_rows(c, _zeros)
        s["dq"], s["dk"], s["dv"] = _split(c, s["grads"])
        ld |= {"lddq": s["dq"].stride(0), "lddk": s["dk"].stride(0), "lddv": s["dv"].stride(0), "lddo": h * d}
    else:
        s["o"] = _zeros((s["q"].shape[0], h * d))
        s["lse"] = _zeros((h, s["q"].shape[0]), torch.float32)
    a = dlo.make_attn_packed(batch=c["batch"], heads=h, kv_heads=c["kv_heads"], head_dim=d, rows_q=s["q"].shape[0],
                             rows_k=s["k"].shape[0], causal_block=c["causal_block"], q_starts=s["q_starts"].data_ptr(),
                             k_starts=s["k_starts"].data_ptr(), **ld)
    size = dlo.dlo_attention_packed_bwd_workspace_bytes if c["op"] == "attn_bwd" else dlo.dlo_attention_packed_fwd_workspace_bytes
    s["attn"], s["ws"] = a, torch.empty(max(size(a), 256), dtype=torch.uint8, device=DEV)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)


def _run_own(s):
    dlo, c, op = _dlo(), s["case"], s["case"]["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "plan":
        dlo.dlo_op_packed_plan(s["grids"].data_ptr(), s["offsets"].data_ptr(), c["batch"], c["axes"], c["rows"] + c["slack"],
                               s["starts"].data_ptr(), s["positions"].data_ptr(), stream)
        return [s["starts"], s["positions"]]
    if op.startswith("rope"):
        call = dlo.dlo_op_rope_fwd if op == "rope_fwd" else dlo.dlo_op_rope_bwd
        call(s["rope"], s["x"].data_ptr(), s["positions"].data_ptr(), s["steps"].data_ptr(), c["rows"], s["y"].data_ptr(), stream)
        return s["y"][:, :c["heads"] * c["head_dim"]]
    if op == "attn_fwd":
        dlo.dlo_op_attention_packed_fwd(s["attn"], s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(),
                                        s["o"].data_ptr(), s["lse"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(),
                                        s["err"].data_ptr(), stream)
        return [s["o"], s["lse"]]
    dlo.dlo_op_attention_packed_bwd(s["attn"], s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(),
                                    s["o"].data_ptr(), s["lse"].data_ptr(), s["do"].data_ptr(), s["dq"].data_ptr(),
                                    s["dk"].data_ptr(), s["dv"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(),
                                    s["err"].data_ptr(), stream)
    return [s["dq"], s["dk"], s["dv"]]


def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plan_plain, "rope_fwd": _rope_plain, "rope_bwd": _rope_plain, "attn_fwd": _attn_fwd_plain,
            "attn_bwd": _attn_bwd_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------ work

def _pairs(case):
    """Visible (query, key) pairs of one head, over all sequences."""
    n, total = case["causal_block"], 0
    for a, b in zip(_q_lengths(case), _k_lengths(case)):
        if not n:
            total += a * b
        else:
            total += sum(min(b, ((i + b - a) // n + 1) * n) for i in range(max(0, a - b), a))
    return total


def work(case):
    op = case["op"]
    if op == "plan":
        return {"bytes": 4 * (2 * case["batch"] * case["axes"] + case["batch"] + 1 + case["rows"] * case["axes"]),
                "flops": 4 * case["rows"] * case["axes"]}
    if op.startswith("rope"):
        n, h = case["rows"], case["heads"]
        return {"bytes": 4 * n * h * case["head_dim"] + 4 * n * case["axes"] + 4 * case["rot"], "flops": 3 * n * h * case["rot"]}
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    rq, rk = sum(_q_lengths(case)), sum(_k_lengths(case))
    q, kv, lse = 2 * rq * h * d, 2 * rk * g * d, 4 * rq * h
    pairs = _pairs(case) * h * d
    if op == "attn_fwd":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs}
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * pairs}


# ------------------------------------------------------------------ in 64 bits

def _exact_plan(s):
    c = s["case"]
    starts, rows = [0], []
    for grid, at in zip(s["host_grids"], s["offsets"].tolist()):
        each = torch.cartesian_prod(*[torch.arange(n) + o for n, o in zip(grid, at)]).view(-1, c["axes"])
        starts.append(starts[-1] + each.shape[0])
        rows.append(each)
    positions = torch.zeros((c["rows"] + c["slack"], c["axes"]), dtype=torch.int32)
    positions[:starts[-1]] = torch.cat(rows)
    return [_int32(starts), positions.to(DEV)]


def _exact_rope(s):
    """As a product of complex numbers, a pair at a time."""
    c = s["case"]
    h, hd, rot = c["heads"], c["head_dim"], c["rot"]
    x = s["x"][:, :h * hd].double().view(-1, h, hd)
    y = x.clone()
    pair = 0
    for a, (dim, base, scaling, factor) in enumerate(_axes(c)):
        at = s["positions"][:, a].double()
        for p in range(dim // 2):
            f = base ** (-2.0 * p / dim)
            if scaling == "base" and dim > 2:
                f *= factor ** (-2.0 * p / (dim - 2))
            if scaling in ("turns", "index"):
                if scaling == "turns":
                    keep = min(1.0, max(0.0, (LENGTH / (2 * math.pi / f) - SLOW) / (FAST - SLOW)))
                else:
                    low, high = (dim / 2 * math.log(LENGTH / (2 * math.pi * t), base) for t in (FAST, SLOW))
                    low, high = max(0, math.floor(low)), min(dim - 1, math.ceil(high))
                    keep = 1 - min(1.0, max(0.0, (p - low) / max(high - low, 0.001)))
                f = keep * f + (1 - keep) * f / factor
            elif scaling == "linear":
                f /= factor
            i, j = (pair, pair + rot // 2) if c["layout"] == "half" else (2 * pair, 2 * pair + 1)
            turn = torch.polar(torch.full_like(at, AMP), at * (f if c["op"] == "rope_fwd" else -f))
            z = torch.complex(x[..., i], x[..., j]) * turn[:, None]
            y[..., i], y[..., j] = z.real, z.imag
            pair += 1
    return y.flatten(1)


def _exact_attention(s):
    """The definition, one head of one sequence at a time; gradients where there is a `do`."""
    c = s["case"]
    h, g, d = c["heads"], c["kv_heads"], c["head_dim"]
    rows, keys = s["q"].shape[0], s["k"].shape[0]
    f64 = {"dtype": torch.float64, "device": DEV}
    o, lse = torch.zeros((rows, h, d), **f64), torch.zeros((h, rows), **f64)
    dq, dk, dv = torch.zeros((rows, h, d), **f64), torch.zeros((keys, g, d), **f64), torch.zeros((keys, g, d), **f64)
    q, k, v = s["q"].unflatten(1, (h, d)), s["k"].unflatten(1, (g, d)), s["v"].unflatten(1, (g, d))
    qs, ks = s["q_starts"].tolist(), s["k_starts"].tolist()
    for b in range(c["batch"]):
        nq, nk = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        lse[:, qs[b]:qs[b + 1]] = -math.inf
        first = max(0, nq - nk) if c["causal_block"] else 0
        if nk == 0 or first >= nq:
            continue
        rq, rk = slice(qs[b] + first, qs[b + 1]), slice(ks[b], ks[b + 1])
        local = torch.arange(first, nq, device=DEV)
        last = torch.full_like(local, nk)             # one past the last key that a query sees
        if c["causal_block"]:
            last = torch.minimum(last, ((local + (nk - nq)) // c["causal_block"] + 1) * c["causal_block"])
        hidden = torch.arange(nk, device=DEV)[None, :] >= last[:, None]
        for m in range(h):
            e = m * g // h
            qq, kk, vv = q[rq, m].double(), k[rk, e].double(), v[rk, e].double()
            x = (qq @ kk.T) / math.sqrt(d)
            x[hidden] = -math.inf
            lse[m, rq] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[m, rq, None])
            o[rq, m] = p @ vv
            if "do" in s:
                do = s["do"].unflatten(1, (h, d))[rq, m].double()
                dv[rk, e] += p.T @ do
                ds = p * (do @ vv.T - (do * o[rq, m]).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[rq, m] = ds @ kk
                dk[rk, e] += ds.T @ qq
    if "do" in s:
        return [dq.flatten(1), dk.flatten(1), dv.flatten(1)]
    return [o.flatten(1), lse]


def exact(case, seed):
    # double-precision products run at about a TFLOP/s here
    if case["op"].startswith("attn") and (10 if case["op"] == "attn_bwd" else 4) * case["heads"] * case["head_dim"] * sum(
            a * b for a, b in zip(_q_lengths(case), _k_lengths(case))) > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    return _exact_rope(s) if case["op"].startswith("rope") else _exact_attention(s)
