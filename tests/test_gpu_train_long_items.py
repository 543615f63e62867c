"""The padded attention's backward pass where dQ's CTAs last longer than the limit of a wait (2 s) on half of the
SMs: dK, dV's CTAs that started on the others wait for their end.  Sums as in the packed operators' test."""
import math

import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

from test_gpu_packed_long_items import DEV, HD, LONG, P, SCALE, SUM, memory_back, near, zeros  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_many_key_tiles():
    heads, nq, nk = 77, 128, LONG * 128
    q, do, k, v = zeros(nq, heads), zeros(nq, heads), zeros(nk, 1), zeros(nk, 1)
    k[::32] = 1.0
    do[...] = 1.0
    v[..., 0] = 1.0
    o, lse = torch.zeros_like(q), torch.full((heads, nq), 7 * math.log(2.0), dtype=torch.float32, device=DEV)
    dq, dk, dv = (torch.full_like(t, 3.5) for t in (q, k, v))
    a = dlo.make_attn(batch=1, heads=heads, kv_heads=1, head_dim=HD, nq=nq, nk=nk, ldq=heads * HD, ldk=HD, ldv=HD, ldo=heads * HD,
                      lddq=heads * HD, lddk=HD, lddv=HD, lddo=heads * HD)
    ws = torch.empty(dlo.dlo_attention_bwd_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dlo.dlo_op_attention_bwd(a, *(t.data_ptr() for t in (q, k, v, o, lse, do, dq, dk, dv)), ws.data_ptr(), ws.numel(), err.data_ptr(),
                             torch.cuda.current_stream().cuda_stream)
    assert int(err.item()) == 0
    assert near(dq, SUM * SCALE)
    assert not bool(dk.any()) and bool((dv == heads * nq * P).all())
