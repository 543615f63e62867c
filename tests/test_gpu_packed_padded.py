"""One sequence in both forms, padded and packed, and the packed form in far rows, each against the plain form in 64 bits
with the packed tests' bounds: scores, P and statistics of the two forms are the same products in the same order, so O,
lse and dV agree bit for bit where neither splits its keys or queries; D is summed otherwise, so dQ and dK agree
within their bounds."""
import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

from test_gpu_packed import DEV, KEEP, Packed, float32_by_default, scratch, stream, within  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cb", [0, 1, 100])
@pytest.mark.parametrize("shape", [(32, 64, 700, 700), (32, 72, 700, 900), (32, 128, 640, 640), (40, 128, 523, 411)], ids=str)
def test_one_sequence_in_both_forms(shape, cb):
    H, hd, nq, nk = shape
    p = Packed(H, H, hd, [nq], [nk], cb)
    p.forward()
    p.backward()
    o, lse = torch.full_like(p.o, KEEP), torch.full_like(p.lse, KEEP)
    g = [torch.full_like(t, KEEP) for t in p.g]
    a = dlo.make_attn(batch=1, heads=H, head_dim=hd, nq=nq, nk=nk, causal_block=cb, ldq=p.q.stride(0), ldk=p.k.stride(0),
                      ldv=p.v.stride(0), ldo=o.stride(0), lddq=g[0].stride(0), lddk=g[1].stride(0), lddv=g[2].stride(0),
                      lddo=p.do.stride(0))
    ws = scratch(max(dlo.dlo_attention_fwd_workspace_bytes(a), dlo.dlo_attention_bwd_workspace_bytes(a)))
    ops = [t.data_ptr() for t in (p.q, p.k, p.v, o, lse)]
    dlo.dlo_op_attention_fwd(a, *ops, ws.data_ptr(), ws.numel(), p.err.data_ptr(), stream())
    dlo.dlo_op_attention_bwd(a, *ops, p.do.data_ptr(), *(t.data_ptr() for t in g), ws.data_ptr(), ws.numel(), p.err.data_ptr(),
                             stream())
    ref = p.reference()
    p.check(ref, grads=True)
    assert torch.equal(o, p.o) and torch.equal(lse, p.lse) and torch.equal(g[2], p.g[2])
    for x, y, name in zip(g, p.g, ("dq", "dk")):
        within(x.unflatten(1, (H, hd)), ref[name], ref[name + "_b"], "padded " + name)
        within(x.unflatten(1, (H, hd)), y.double().unflatten(1, (H, hd)), 2 * ref[name + "_b"], "padded and packed " + name)


@pytest.mark.parametrize("hd,far", [(64, 256 * 1100), (72, 256 * 1100 + 77), (128, 256 * 1100 + 5)])
def test_far_rows_within_the_bounds_of_near_ones(hd, far):
    """281600 rows of 8192 elements before the sequences: offsets past 2^31."""
    p = Packed(2, 1, hd, [200, 0, 131], None, 1, lead=far, slack=3, pad=8192 - 4 * hd)
    assert p.q.stride(0) * far > 2 ** 31
    ref = p.reference()
    p.forward()
    p.backward()
    p.check(ref, grads=True)
    del p, ref
    torch.cuda.empty_cache()
