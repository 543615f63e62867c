"""Device int32 operands of the training attention (lengths, error word) that are not on a
4-byte boundary would fault where a kernel reads them: refused before any launch
(no GPU needed: addresses are never read)."""
import pytest

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

P = 1 << 20            # an aligned address that nothing reads
BIG = 1 << 60


@pytest.mark.parametrize("kw,err", [(dict(q_lens=P + 2), P), (dict(k_lens=P + 1), P), (dict(), P + 2)])
def test_int32_operands_off_their_boundary_are_refused(kw, err):
    a = dlo.make_attn(batch=2, heads=4, kv_heads=2, head_dim=64, nq=100, nk=200, ldq=256, ldk=128, ldv=128, ldo=256, lddq=256,
                      lddk=128, lddv=128, lddo=256, **kw)
    for call in (lambda: dlo.dlo_op_attention_fwd(a, P, P, P, P, P, P, BIG, err, None),
                 lambda: dlo.dlo_op_attention_bwd(a, P, P, P, P, P, P, P, P, P, P, BIG, err, None)):
        with pytest.raises(dlo.DloError) as e:
            call()
        assert e.value.status == dlo.EINVAL and str(e.value)
