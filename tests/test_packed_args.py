"""Operators for packed batches, without a GPU: refusals and workspace sizes, checked
before any launch (addresses are never read), and the table of rotary steps."""
import ctypes
import math

import numpy as np
import pytest

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

P = 1 << 20            # an aligned address that nothing reads
BIG = 1 << 60


def attn(**kw):
    base = dict(batch=3, heads=4, kv_heads=2, head_dim=64, rows_q=100, rows_k=200, causal_block=0, ldq=256, ldk=128, ldv=128,
                ldo=256, lddq=256, lddk=128, lddv=128, lddo=256, q_starts=P, k_starts=P)
    return dlo.make_attn_packed(**{**base, **kw})


def refused(status, f, *a):
    with pytest.raises(dlo.DloError) as e:
        f(*a)
    assert e.value.status == status and str(e.value)


@pytest.mark.parametrize("kw", [dict(batch=0), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(rows_q=0), dict(rows_k=0),
                                dict(head_dim=12), dict(head_dim=136), dict(head_dim=0), dict(causal_block=-1),
                                dict(batch=65536), dict(rows_q=-5), dict(rows_q=(1 << 30) + 1), dict(rows_k=(1 << 30) + 1),
                                dict(heads=65536)])
def test_attention_descriptions_are_refused(kw):
    a = attn(**kw)
    refused(dlo.EINVAL, dlo.dlo_attention_packed_fwd_workspace_bytes, a)
    refused(dlo.EINVAL, dlo.dlo_attention_packed_bwd_workspace_bytes, a)
    refused(dlo.EINVAL, dlo.dlo_op_attention_packed_fwd, a, P, P, P, P, P, P, BIG, None, None)
    refused(dlo.EINVAL, dlo.dlo_op_attention_packed_bwd, a, P, P, P, P, P, P, P, P, P, P, BIG, None, None)


@pytest.mark.parametrize("kw", [dict(ldq=252), dict(ldq=248), dict(ldk=120), dict(ldv=132), dict(ldo=0), dict(q_starts=None),
                                dict(k_starts=None), dict(q_starts=P + 2), dict(k_starts=P + 1)])
def test_attention_operand_layouts_are_refused(kw):
    a = attn(**kw)
    refused(dlo.EINVAL, dlo.dlo_op_attention_packed_fwd, a, P, P, P, P, P, P, BIG, None, None)
    refused(dlo.EINVAL, dlo.dlo_op_attention_packed_bwd, a, P, P, P, P, P, P, P, P, P, P, BIG, None, None)


@pytest.mark.parametrize("kw", [dict(lddq=128), dict(lddk=12), dict(lddv=0), dict(lddo=-256)])
def test_attention_gradient_strides_are_refused(kw):
    refused(dlo.EINVAL, dlo.dlo_op_attention_packed_bwd, attn(**kw), P, P, P, P, P, P, P, P, P, P, BIG, None, None)


def test_attention_operands_are_refused():
    a = attn()
    for n, call in ((5, dlo.dlo_op_attention_packed_fwd), (9, dlo.dlo_op_attention_packed_bwd)):
        for i in range(n):
            for bad in (None, P + 2):
                args = [P] * n
                args[i] = bad
                refused(dlo.EINVAL, call, a, *args, P, BIG, None, None)
        size = (dlo.dlo_attention_packed_fwd_workspace_bytes if n == 5 else dlo.dlo_attention_packed_bwd_workspace_bytes)(a)
        refused(dlo.ENOMEM, call, a, *[P] * n, P, size - 1, None, None)
        refused(dlo.EINVAL, call, a, *[P] * n, None, size, None, None)
        refused(dlo.EINVAL, call, a, *[P] * n, P + 16, size, None, None)
        refused(dlo.EINVAL, call, a, *[P] * n, P, size, P + 2, None)


@pytest.mark.parametrize("kw", [dict(grids=None), dict(starts=None), dict(batch=0), dict(batch=65536), dict(axes=0), dict(axes=5),
                                dict(rows=0), dict(rows=(1 << 30) + 1), dict(grids=P + 2), dict(offsets=P + 1), dict(starts=P + 3),
                                dict(positions=P + 2)])
def test_plan_refusals(kw):
    base = dict(grids=P, offsets=P, batch=2, axes=3, rows=10, starts=P, positions=P)
    refused(dlo.EINVAL, dlo.dlo_op_packed_plan, *{**base, **kw}.values(), None)


AXIS = dict(dim=32, theta=10000.0)
BY = dict(dim=32, scaling=dlo.ROPE_BY_TURNS, factor=4.0, length=1000.0)
NAN, INF = float("nan"), float("inf")


def rope(**kw):
    return dlo.make_rope(**{**dict(heads=3, head_dim=64, axes=[AXIS, AXIS], ldx=192, ldy=200), **kw})


@pytest.mark.parametrize("kw", [dict(heads=0), dict(heads=65536), dict(head_dim=60), dict(head_dim=0), dict(head_dim=264),
                                dict(layout=2), dict(layout=-1), dict(axes=[]), dict(axes=[dict(dim=2)] * 5), dict(amp=NAN), dict(amp=INF),
                                dict(axes=[dict(dim=0)]), dict(axes=[dict(dim=-2)]), dict(axes=[dict(dim=7)]), dict(axes=[dict(dim=66)]),
                                dict(axes=[dict(dim=34), AXIS]), dict(axes=[dict(dim=8, theta=1.0)]), dict(axes=[dict(dim=8, theta=NAN)]),
                                dict(axes=[dict(dim=8, theta=INF)]), dict(axes=[dict(dim=8, scaling=5)]), dict(axes=[dict(dim=8, scaling=-1)]),
                                dict(axes=[dict(dim=8, scaling=1, factor=0.5)]), dict(axes=[dict(dim=8, scaling=2, factor=NAN)]),
                                dict(axes=[{**BY, "length": 0.0}]), dict(axes=[{**BY, "slow": 0.0}]),
                                dict(axes=[{**BY, "fast": 1.0}]), dict(axes=[{**BY, "scaling": dlo.ROPE_BY_INDEX, "fast": INF}])])
def test_rope_descriptions_are_refused(kw):
    r = rope(**kw)
    refused(dlo.EINVAL, dlo.dlo_rope_steps, r)
    refused(dlo.EINVAL, dlo.dlo_op_rope_fwd, r, P, P, P, 4, P, None)
    refused(dlo.EINVAL, dlo.dlo_op_rope_bwd, r, P, P, P, 4, P, None)


@pytest.mark.parametrize("call", [dlo.dlo_op_rope_fwd, dlo.dlo_op_rope_bwd])
def test_rope_operands_are_refused(call):
    good = dict(x=P, positions=P, steps=P, rows=4, y=P + 4096)
    for kw in (dict(x=None), dict(positions=None), dict(steps=None), dict(y=None), dict(rows=0), dict(rows=(1 << 30) + 1),
               dict(x=P + 8), dict(positions=P + 2), dict(steps=P + 4), dict(y=P + 8), dict(y=P)):       # in place, other strides
        refused(dlo.EINVAL, call, rope(), *{**good, **kw}.values(), None)
    for kw in (dict(ldx=184), dict(ldx=196), dict(ldy=0), dict(ldy=-200)):
        refused(dlo.EINVAL, call, rope(**kw), *good.values(), None)


def test_rope_steps_are_the_frequencies():
    """Against the formulas in Python's own floats: some ten roundings of 2^-53, enlarged up to 40 times by the exponent
    of pow and the difference under keep, are below 1e-13; and a step is rounded to a whole number, half of 2^-64."""
    length, fast, slow, factor = 4096.0, 32.0, 1.0, 8.0
    for scaling in range(5):
        for dim, theta in ((2, 10000.0), (44, 10000.0), (128, 500000.0)):
            r = rope(head_dim=256, ldx=768, ldy=768, axes=[dict(dim=16), dict(dim=dim, theta=theta, scaling=scaling, factor=factor,
                                                                                 length=length, fast=fast, slow=slow)])
            steps = dlo.dlo_rope_steps(r).view(np.uint64)
            assert steps.shape == (8 + dim // 2,)
            base = theta * factor ** (dim / (dim - 2)) if scaling == dlo.ROPE_BASE and dim > 2 else theta
            at = [dim * math.log(length / (2 * math.pi * t)) / (2 * math.log(base)) for t in (fast, slow)]
            low, high = max(0, math.floor(at[0])), min(dim - 1, math.ceil(at[1]))
            for p in range(dim // 2):
                f = base ** (-2 * p / dim)
                keep = {dlo.ROPE_PLAIN: 1.0, dlo.ROPE_LINEAR: 0.0, dlo.ROPE_BASE: 1.0,
                        dlo.ROPE_BY_TURNS: min(1.0, max(0.0, (length * f / (2 * math.pi) - slow) / (fast - slow))),
                        dlo.ROPE_BY_INDEX: 1 - min(1.0, max(0.0, (p - low) / max(high - low, 1e-3)))}[scaling]
                want = f * (keep + (1 - keep) / factor) / (2 * math.pi)
                assert abs(int(steps[8 + p]) / 2.0 ** 64 - want) <= 1e-13 * want + 2.0 ** -65, (scaling, dim, p)


def test_rope_steps_want_their_number():
    r = rope()
    steps = (ctypes.c_ulonglong * 64)()
    assert dlo._c["dlo_rope_steps"](ctypes.byref(r), steps, 31) == dlo.EINVAL
    assert dlo._c["dlo_rope_steps"](ctypes.byref(r), None, 32) == dlo.EINVAL
    assert dlo._c["dlo_rope_steps"](ctypes.byref(r), steps, 32) == dlo.OK


def test_workspaces_grow_with_the_problem():
    # row statistics of every slot, and partial results only where few query rows share long keys
    assert dlo.dlo_attention_packed_bwd_workspace_bytes(attn()) >= 4 * 3 * 128 * 32
    few = attn(batch=1, rows_q=1, rows_k=100000)
    assert dlo.dlo_attention_packed_fwd_workspace_bytes(few) > dlo.dlo_attention_packed_fwd_workspace_bytes(attn(rows_q=100000))


def packed_tile(starts, batch, rows, t, slot):
    """The kernels' search for the tile of a slot, a lane at a time (attention.cuh: packed_tile)."""
    at = lambda b: min(max(starts[b], 0), rows)          # noqa: E731
    b, n = 0, batch
    while True:
        step = (n + 30) // 31
        index = [b + min(lane * step, n) for lane in range(32)]
        assert all(0 <= i <= batch for i in index)
        before = [lane for lane in range(32) if lane * step < n and at(index[lane]) // t + index[lane] <= slot]
        k = before[-1] if before else 0
        if step == 1:
            row0, end = at(index[k]), at(index[k + 1])
            b += k
            break
        b += k * step
        n = min(step, n - k * step)
    tile = slot - (row0 // t + b)
    return (b, tile if tile * t < max(0, end - row0) else -1)


@pytest.mark.parametrize("t", [128, 25, 1])
def test_every_tile_of_every_sequence_has_one_slot(t):
    rng = np.random.default_rng(t)
    for batch in (1, 2, 31, 32, 33, 64, 65, 700, 2100):
        for lead, mean in ((0, 2 * t), (5 * t + 3, t // 2 + 1)):
            lens = rng.integers(0, 2 * mean + 1, batch) * (rng.random(batch) < 0.8)
            starts = np.concatenate([[lead], lead + np.cumsum(lens)]).tolist()
            rows = starts[-1] + 7
            want = {(b, i) for b in range(batch) for i in range((starts[b + 1] - starts[b] + t - 1) // t)}
            found = [packed_tile(starts, batch, rows, t, s) for s in range(rows // t + batch)]
            found = [f for f in found if f[1] >= 0]
            assert len(found) == len(want) and set(found) == want, (t, batch, lead)
