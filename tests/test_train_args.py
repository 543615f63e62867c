"""Refusals and workspace sizes of the training ops, checked before any launch
(no GPU needed: addresses are never read)."""
import pytest

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

P = 1 << 20            # an aligned address that nothing reads
BIG = 1 << 60


def attn(**kw):
    base = dict(batch=2, heads=4, kv_heads=2, head_dim=64, nq=100, nk=200, causal_block=0, ldq=256, ldk=128, ldv=128,
                ldo=256, lddq=256, lddk=128, lddv=128, lddo=256)
    return dlo.make_attn(**{**base, **kw})


def refused(status, f, *a):
    with pytest.raises(dlo.DloError) as e:
        f(*a)
    assert e.value.status == status and str(e.value)


@pytest.mark.parametrize("kw", [dict(batch=0), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(nq=0), dict(nk=0),
                                dict(head_dim=12), dict(head_dim=136), dict(head_dim=0), dict(causal_block=-1),
                                dict(batch=70000), dict(nq=-5), dict(batch=60000, nq=1 << 20), dict(heads=65536)])
def test_attention_descriptions_are_refused(kw):
    a = attn(**kw)
    refused(dlo.EINVAL, dlo.dlo_attention_fwd_workspace_bytes, a)
    refused(dlo.EINVAL, dlo.dlo_attention_bwd_workspace_bytes, a)
    refused(dlo.EINVAL, dlo.dlo_op_attention_fwd, a, P, P, P, P, P, P, BIG, None, None)
    refused(dlo.EINVAL, dlo.dlo_op_attention_bwd, a, P, P, P, P, P, P, P, P, P, P, BIG, None, None)


@pytest.mark.parametrize("kw", [dict(ldq=252), dict(ldq=248), dict(ldk=120), dict(ldv=132), dict(ldo=0)])
def test_attention_strides_are_refused(kw):
    a = attn(**kw)
    refused(dlo.EINVAL, dlo.dlo_op_attention_fwd, a, P, P, P, P, P, P, BIG, None, None)
    refused(dlo.EINVAL, dlo.dlo_op_attention_bwd, a, P, P, P, P, P, P, P, P, P, P, BIG, None, None)


@pytest.mark.parametrize("kw", [dict(lddq=128), dict(lddk=12), dict(lddv=0), dict(lddo=-256)])
def test_attention_gradient_strides_are_refused(kw):
    refused(dlo.EINVAL, dlo.dlo_op_attention_bwd, attn(**kw), P, P, P, P, P, P, P, P, P, P, BIG, None, None)


def test_attention_operands_are_refused():
    a = attn()
    for i in range(5):
        for bad in (None, P + 2):
            args = [P] * 5
            args[i] = bad
            refused(dlo.EINVAL, dlo.dlo_op_attention_fwd, a, *args, P, BIG, None, None)
    for i in range(9):
        for bad in (None, P + 2):
            args = [P] * 9
            args[i] = bad
            refused(dlo.EINVAL, dlo.dlo_op_attention_bwd, a, *args, P, BIG, None, None)
    fwd, bwd = dlo.dlo_attention_fwd_workspace_bytes(a), dlo.dlo_attention_bwd_workspace_bytes(a)
    refused(dlo.ENOMEM, dlo.dlo_op_attention_fwd, a, *[P] * 5, P, fwd - 1, None, None)
    refused(dlo.ENOMEM, dlo.dlo_op_attention_bwd, a, *[P] * 9, P, bwd - 1, None, None)
    refused(dlo.EINVAL, dlo.dlo_op_attention_bwd, a, *[P] * 9, None, bwd, None, None)
    refused(dlo.EINVAL, dlo.dlo_op_attention_bwd, a, *[P] * 9, P + 16, bwd, None, None)


def test_attention_workspaces_grow_with_the_problem():
    # two statistics a query row, and partial results only where few query tiles share long keys
    assert dlo.dlo_attention_bwd_workspace_bytes(attn()) >= 2 * 4 * 100 * 8
    few = attn(batch=1, nq=1, nk=100000)
    assert dlo.dlo_attention_fwd_workspace_bytes(few) > dlo.dlo_attention_fwd_workspace_bytes(attn(nq=100000, nk=64))


LN = dict(x=P, rows=10, D=64, rpb=5, shift=None, scale=None, mod_ld=64, w=None, b=None, eps=1e-6, out=P, mean=P, rstd=P)


@pytest.mark.parametrize("kw", [dict(x=None), dict(out=None), dict(mean=None), dict(rstd=None), dict(rows=0), dict(D=6), dict(D=0),
                                dict(D=20484), dict(rpb=0), dict(shift=P), dict(w=P), dict(shift=P, scale=P, w=P, b=P),
                                dict(shift=P, scale=P, mod_ld=60), dict(shift=P, scale=P, mod_ld=66), dict(shift=P, scale=P + 4),
                                dict(eps=0.0), dict(eps=float("nan")), dict(x=P + 4), dict(rows=(1 << 30) + 1)])
def test_layernorm_fwd_refusals(kw):
    refused(dlo.EINVAL, dlo.dlo_op_layernorm_fwd, *{**LN, **kw}.values(), None)


LNB = dict(dy=P, x=P, mean=P, rstd=P, rows=10, D=64, rpb=5, scale=P, mod_ld=64, w=None, dres=None, dx=P, dshift=P, dscale=P,
           dmod_ld=64, ws=P, ws_bytes=BIG)


@pytest.mark.parametrize("kw,status", [(dict(dy=None), -1), (dict(x=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
                                       (dict(dx=None), -1), (dict(rows=0), -1), (dict(D=6), -1), (dict(D=20484), -1),
                                       (dict(rpb=0), -1), (dict(w=P), -1), (dict(dshift=None), -1), (dict(scale=None), -1),
                                       (dict(mod_ld=60), -1), (dict(dmod_ld=60), -1), (dict(dmod_ld=66), -1), (dict(dx=P + 4), -1),
                                       (dict(dres=P + 4), -1), (dict(dy=P + 2), -1), (dict(ws=None), -1), (dict(ws_bytes=255), -3)])
def test_layernorm_bwd_refusals(kw, status):
    refused(status, dlo.dlo_op_layernorm_bwd, *{**LNB, **kw}.values(), None)


RMB = dict(dy=P, lddy=64, x=P, ldx=64, w=P, rstd=P, rows=10, D=64, dx=P + 4096, lddx=64, dw=P, ws=P, ws_bytes=BIG)


@pytest.mark.parametrize("kw,status", [(dict(dy=None), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(rstd=None), -1),
                                       (dict(dx=None), -1), (dict(rows=0), -1), (dict(D=12), -1), (dict(D=20488), -1),
                                       (dict(lddy=56), -1), (dict(ldx=68), -1), (dict(lddx=60), -1), (dict(dx=P, lddx=72), -1),
                                       (dict(dx=P + 4104), -1), (dict(ws=None), -1), (dict(ws_bytes=15), -3)])
def test_rmsnorm_bwd_refusals(kw, status):
    refused(status, dlo.dlo_op_rmsnorm_bwd, *{**RMB, **kw}.values(), None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(w=None), dict(y=None), dict(rstd=None), dict(rows=0), dict(D=12), dict(ldx=56),
                                dict(ldy=60), dict(eps=-1.0), dict(y=P + 8)])
def test_rmsnorm_fwd_refusals(kw):
    base = dict(x=P, ldx=64, rows=10, D=64, w=P, eps=1e-6, y=P, ldy=64, rstd=P)
    refused(dlo.EINVAL, dlo.dlo_op_rmsnorm_fwd, *{**base, **kw}.values(), None)


def test_norm_workspace_sizes_are_refused():
    for rows, d, rpb in ((0, 64, 1), (1, 6, 1), (1, 20484, 1), (1, 64, 0)):
        refused(dlo.EINVAL, dlo.dlo_layernorm_bwd_workspace_bytes, rows, d, rpb)
    for rows, d in ((0, 64), (1, 12), (1, 20488)):
        refused(dlo.EINVAL, dlo.dlo_rmsnorm_bwd_workspace_bytes, rows, d)
