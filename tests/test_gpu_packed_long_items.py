"""Packed attention's backward pass where one item of a CTA lasts longer than the limit of a wait (2 s):
the waits of its warps are for steps, of which such an item has three million.  The values are such that every sum
is exact in fp32: P = 2^-7, and one row in 32 counts, 12.6 million in all."""
import math

import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
HD = 8
LONG = 3 << 20                       # steps
P = 2.0 ** -7
SUM = LONG * 128 / 32 * P            # 98304, exact in bf16
SCALE = 1 / math.sqrt(HD)


def zeros(rows, heads):
    return torch.zeros((rows, heads, HD), dtype=torch.bfloat16, device=DEV)


def backward(heads, nq, nk, q, k, v, do):
    """With one key/value head, O = 0 and P = 2^-7 everywhere (scores are 0)."""
    o, lse = torch.zeros_like(q), torch.full((heads, nq), 7 * math.log(2.0), dtype=torch.float32, device=DEV)
    g = [torch.full_like(t, 3.5) for t in (q, k, v)]
    qs, ks = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (nq, nk))
    a = dlo.make_attn_packed(batch=1, heads=heads, kv_heads=1, head_dim=HD, rows_q=nq, rows_k=nk, ldq=heads * HD, ldk=HD, ldv=HD,
                             ldo=heads * HD, lddq=heads * HD, lddk=HD, lddv=HD, lddo=heads * HD, q_starts=qs.data_ptr(),
                             k_starts=ks.data_ptr())
    ws = torch.empty(dlo.dlo_attention_packed_bwd_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dlo.dlo_op_attention_packed_bwd(a, *(t.data_ptr() for t in (q, k, v, o, lse, do, *g)), ws.data_ptr(), ws.numel(), err.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream)
    assert int(err.item()) == 0
    return g


@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def near(y, want):
    return bool(((y.double() - want).abs() <= 2.0 ** -8 * want).all())


def test_many_query_tiles_of_many_heads():
    """dK, dV: 128 heads of 24576 query tiles to each of 76 key tiles."""
    heads, nq, nk = 128, LONG, 76 * 128
    q, do, k, v = zeros(nq, heads), zeros(nq, heads), zeros(nk, 1), zeros(nk, 1)
    q[::32] = 1.0
    do[::32] = 1.0
    v[..., 0] = 1.0                  # dP = 1 in the rows that count
    dq, dk, dv = backward(heads, nq, nk, q, k, v, do)
    assert not bool(dq.any())
    assert bool((dv == SUM).all()) and near(dk, SUM * SCALE)


def test_many_key_tiles():
    """dQ: 77 heads of one query tile over 3145728 key tiles, the last one not full.  Half of the SMs have none of
    them, and dK, dV's CTAs there wait for the others' end."""
    heads, nq, nk = 77, 128, LONG * 128 - 28
    q, do, k, v = zeros(nq, heads), zeros(nq, heads), zeros(nk, 1), zeros(nk, 1)
    k[::32] = 1.0
    do[...] = 1.0
    v[..., 0] = 1.0
    dq, dk, dv = backward(heads, nq, nk, q, k, v, do)
    assert near(dq, SUM * SCALE)
    assert not bool(dk.any()) and bool((dv == heads * nq * P).all())
