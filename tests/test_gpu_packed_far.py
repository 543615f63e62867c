"""Operators for packed batches where offsets pass 2^31 elements: far rows of a large buffer, against the same
rows at the start of a small one, bit for bit (the same tiles: starts that are multiples of 128 and 5 apart)."""
import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.fixture(autouse=True)
def float32_by_default():
    """Another test module of the same process may have set another default."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


@pytest.mark.parametrize("hd,far", [(64, 256 * 1100), (128, 256 * 1100 + 5)])
def test_attention_of_far_rows(hd, far):
    H, G, lens, ld = 2, 1, [200, 0, 131], 8192          # 281600 rows of 8192: 2.3e9 elements a matrix
    n = sum(lens)
    g = torch.Generator(device=DEV).manual_seed(3)
    small = [(torch.randn((n, ld), generator=g, device=DEV)).to(torch.bfloat16) for _ in range(4)]
    out = {}
    for first in (0, far):
        rows = first + n
        q, k, v, do = (torch.empty((rows, ld), dtype=torch.bfloat16, device=DEV) for _ in range(4))
        for t, s in zip((q, k, v, do), small):
            t[first:] = s
        grads = [torch.zeros((rows, ld), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        o, lse = torch.zeros((rows, ld), dtype=torch.bfloat16, device=DEV), torch.zeros((H, rows), dtype=torch.float32, device=DEV)
        starts = torch.tensor([first, first + 200, first + 200, first + n], dtype=torch.int32, device=DEV)
        a = dlo.make_attn_packed(batch=3, heads=H, kv_heads=G, head_dim=hd, rows_q=rows, rows_k=rows, causal_block=1, ldq=ld, ldk=ld,
                                 ldv=ld, ldo=ld, lddq=ld, lddk=ld, lddv=ld, lddo=ld, q_starts=starts.data_ptr(), k_starts=starts.data_ptr())
        ws = torch.empty(max(dlo.dlo_attention_packed_fwd_workspace_bytes(a), dlo.dlo_attention_packed_bwd_workspace_bytes(a)),
                         dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ops = [t.data_ptr() for t in (q, k, v, o, lse)]
        dlo.dlo_op_attention_packed_fwd(a, *ops, ws.data_ptr(), ws.numel(), err.data_ptr(), stream())
        dlo.dlo_op_attention_packed_bwd(a, *ops, do.data_ptr(), *(t.data_ptr() for t in grads), ws.data_ptr(), ws.numel(), err.data_ptr(),
                                        stream())
        assert int(err.item()) == 0
        out[first] = [t[first:].clone() for t in [o] + grads] + [lse[:, first:].clone()]
        assert all(not bool(t[max(0, first - 4000):first].any()) for t in [o] + grads)
        del q, k, v, do, grads, o, lse, ws
        torch.cuda.empty_cache()
    widths = (H * hd, H * hd, G * hd, G * hd, n)
    for x, y, w in zip(out[0], out[far], widths):
        # two heads share a tile in the small problem and in the large one; sums of a split gradient may be parted
        # otherwise: bf16 results within a step of each other
        d = (x[:, :w].float() - y[:, :w].float()).abs()
        assert bool((d <= 2.0 ** -6 * y[:, :w].float().abs() + 2.0 ** -7 * y[:, :w].float().abs().max()).all())


def test_rope_of_far_rows():
    heads, hd, ld, rows = 1, 128, 8192, 280000
    x = torch.zeros((rows, ld), dtype=torch.bfloat16, device=DEV)
    tail = torch.randn((300, hd), device=DEV).to(torch.bfloat16)
    x[-300:, :hd] = tail
    positions = torch.arange(rows, device=DEV, dtype=torch.int32)
    r = dlo.make_rope(heads=heads, head_dim=hd, axes=[dict(dim=hd)], ldx=ld, ldy=hd, layout=dlo.ROPE_HALF)
    steps = torch.from_numpy(dlo.dlo_rope_steps(r)).to(DEV)
    y = torch.empty((rows, hd), dtype=torch.bfloat16, device=DEV)
    dlo.dlo_op_rope_fwd(r, x.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, y.data_ptr(), stream())
    r.ldx = hd
    z = torch.empty((300, hd), dtype=torch.bfloat16, device=DEV)
    dlo.dlo_op_rope_fwd(r, tail.data_ptr(), positions[-300:].data_ptr(), steps.data_ptr(), 300, z.data_ptr(), stream())
    assert torch.equal(y[-300:], z) and not bool(y[:1000].any())
