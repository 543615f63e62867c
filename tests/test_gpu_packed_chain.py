"""The operators for packed batches as a training program uses them: half a block over a
packed batch, forward and back, against torch autograd in 64 bits; the same captured into a
graph whose grids change in place; two streams and two threads at once."""
import math
import threading

import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

pytestmark = pytest.mark.gpu

DEV = "cuda"
H, G, HD = 4, 2, 72
W = (H + 2 * G) * HD
AXES = [dict(dim=24, theta=1000.0), dict(dim=24, theta=1000.0), dict(dim=24, theta=1000.0)]


@pytest.fixture(autouse=True)
def float32_by_default():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


class Program:
    """Buffers of one packed batch of `rows` rows at most: plan, q/k norm, rotary positions, attention, and back."""

    def __init__(self, grids, rows, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)               # noqa: E731
        f32 = lambda *s: torch.zeros(s, device=DEV)                                    # noqa: E731
        self.batch, self.rows = len(grids), rows
        self.grids = torch.tensor(grids, dtype=torch.int32, device=DEV)
        self.starts = torch.zeros(self.batch + 1, dtype=torch.int32, device=DEV)
        self.positions = torch.zeros((rows, 3), dtype=torch.int32, device=DEV)
        self.x = torch.randn((rows, W), generator=g, device=DEV).to(torch.bfloat16)
        self.wq = (1 + 0.1 * torch.randn(H * HD, generator=g, device=DEV)).to(torch.bfloat16)
        self.wk = (1 + 0.1 * torch.randn(G * HD, generator=g, device=DEV)).to(torch.bfloat16)
        self.do = (0.1 * torch.randn((rows, H * HD), generator=g, device=DEV)).to(torch.bfloat16)
        self.qkv, self.dqkv, self.dx = bf(rows, W), bf(rows, W), bf(rows, W)
        self.rq, self.rk = f32(rows), f32(rows)
        self.o, self.lse = bf(rows, H * HD), f32(H, rows)
        self.dwq, self.dwk = f32(H * HD), f32(G * HD)
        self.rope = dlo.make_rope(heads=H + G, head_dim=HD, axes=AXES, ldx=W, ldy=W)
        self.steps = torch.from_numpy(dlo.dlo_rope_steps(self.rope)).to(DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.attn = dlo.make_attn_packed(batch=self.batch, heads=H, kv_heads=G, head_dim=HD, rows_q=rows, rows_k=rows, causal_block=5,
                                         ldq=W, ldk=W, ldv=W, ldo=H * HD, lddq=W, lddk=W, lddv=W, lddo=H * HD,
                                         q_starts=self.starts.data_ptr(), k_starts=self.starts.data_ptr())
        need = max(dlo.dlo_attention_packed_fwd_workspace_bytes(self.attn), dlo.dlo_attention_packed_bwd_workspace_bytes(self.attn),
                   dlo.dlo_rmsnorm_bwd_workspace_bytes(rows, H * HD), dlo.dlo_rmsnorm_bwd_workspace_bytes(rows, G * HD))
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)

    def run(self):
        st, n = torch.cuda.current_stream().cuda_stream, self.rows
        at = lambda t, col: t[:, col:].data_ptr()                                      # noqa: E731
        q, k, v = 0, H * HD, (H + G) * HD
        dlo.dlo_op_packed_plan(self.grids.data_ptr(), None, self.batch, 3, n, self.starts.data_ptr(), self.positions.data_ptr(), st)
        dlo.dlo_op_rmsnorm_fwd(at(self.x, q), W, n, H * HD, self.wq.data_ptr(), 1e-6, at(self.qkv, q), W, self.rq.data_ptr(), st)
        dlo.dlo_op_rmsnorm_fwd(at(self.x, k), W, n, G * HD, self.wk.data_ptr(), 1e-6, at(self.qkv, k), W, self.rk.data_ptr(), st)
        self.qkv[:, v:].copy_(self.x[:, v:])
        dlo.dlo_op_rope_fwd(self.rope, self.qkv.data_ptr(), self.positions.data_ptr(), self.steps.data_ptr(), n, self.qkv.data_ptr(), st)
        ws = (self.ws.data_ptr(), self.ws.numel())
        ops = (at(self.qkv, q), at(self.qkv, k), at(self.qkv, v), self.o.data_ptr(), self.lse.data_ptr())
        dlo.dlo_op_attention_packed_fwd(self.attn, *ops, *ws, self.err.data_ptr(), st)
        dlo.dlo_op_attention_packed_bwd(self.attn, *ops, self.do.data_ptr(), at(self.dqkv, q), at(self.dqkv, k), at(self.dqkv, v), *ws,
                                        self.err.data_ptr(), st)
        dlo.dlo_op_rope_bwd(self.rope, self.dqkv.data_ptr(), self.positions.data_ptr(), self.steps.data_ptr(), n, self.dqkv.data_ptr(), st)
        self.dx[:, v:].copy_(self.dqkv[:, v:])
        dlo.dlo_op_rmsnorm_bwd(at(self.dqkv, q), W, at(self.x, q), W, self.wq.data_ptr(), self.rq.data_ptr(), n, H * HD, at(self.dx, q), W,
                               self.dwq.data_ptr(), *ws, st)
        dlo.dlo_op_rmsnorm_bwd(at(self.dqkv, k), W, at(self.x, k), W, self.wk.data_ptr(), self.rk.data_ptr(), n, G * HD, at(self.dx, k), W,
                               self.dwk.data_ptr(), *ws, st)

    def outputs(self):
        return [self.starts, self.positions, self.o, self.lse, self.dx, self.dwq, self.dwk]

    def clear(self):
        """What lies behind the sequences keeps what it holds: zeros, so that the norms' column sums see none of it."""
        for t in self.outputs() + [self.dqkv]:
            t.zero_()


def reference(p):
    """O, dx, dwq, dwk of the valid rows by autograd in 64 bits."""
    grids = p.grids.tolist()
    x = p.x.double().requires_grad_()
    wq, wk = p.wq.double().requires_grad_(), p.wk.double().requires_grad_()
    norm = lambda t, w: t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w     # noqa: E731
    f = torch.cat([torch.tensor(a["theta"], dtype=torch.float64, device=DEV) **
                   (-2 * torch.arange(a["dim"] // 2, dtype=torch.float64, device=DEV) / a["dim"]) for a in AXES])
    axis = [i for i, a in enumerate(AXES) for _ in range(a["dim"] // 2)]

    def turn(t, at):
        t = t.unflatten(1, (-1, HD // 2, 2))
        c, s = (at[:, axis] * f).cos()[:, None], (at[:, axis] * f).sin()[:, None]
        return torch.stack([t[..., 0] * c - t[..., 1] * s, t[..., 0] * s + t[..., 1] * c], -1).flatten(2)

    outs, first = [], 0
    for grid in grids:
        n = math.prod(grid)
        rows = slice(first, first + n)
        first += n
        at = torch.cartesian_prod(*[torch.arange(e, device=DEV) for e in grid]).view(-1, 3).double()
        q = turn(norm(x[rows, :H * HD], wq), at).transpose(0, 1)
        k = turn(norm(x[rows, H * HD:(H + G) * HD], wk), at).transpose(0, 1).repeat_interleave(H // G, 0)
        v = x[rows, (H + G) * HD:].unflatten(1, (G, HD)).transpose(0, 1).repeat_interleave(H // G, 0)
        i = torch.arange(n, device=DEV)
        s = (q @ k.transpose(1, 2) / math.sqrt(HD)).masked_fill((i[:, None] // 5 < i[None] // 5)[None], -math.inf)
        outs.append((torch.softmax(s, -1) @ v).transpose(0, 1).flatten(1))
    o = torch.cat(outs)
    o.backward(p.do[:first].double())
    return o.detach(), x.grad[:first], wq.grad, wk.grad, first


def check(p):
    """In the 2-norm.  A bf16 rounding is off by 2^-9 of the value at most on average over its binade (2^-8 at
    its low end), and q, k (norm, rotation), P, dS, O, its use in D, dq, dk (two ops) are rounded one after the
    other: some eight roundings of independent sign, sqrt(8) 2^-9 = 5.5e-3, taken twice."""
    o, dx, dwq, dwk, n = reference(p)
    assert int(p.err.item()) == 0
    for name, y, want in (("o", p.o[:n], o), ("dx", p.dx[:n], dx), ("dwq", p.dwq, dwq), ("dwk", p.dwk, dwk)):
        err = float((y.double() - want).norm() / want.norm())
        assert err <= 1.1e-2, (name, err)


GRIDS = [[2, 5, 7], [1, 1, 1], [3, 9, 10], [0, 4, 4], [1, 16, 16]]
OTHERS = [[5, 9, 9], [2, 2, 2], [1, 1, 1], [1, 10, 20], [0, 0, 0]]


def test_half_a_block_of_a_packed_batch():
    p = Program(GRIDS, 700)
    p.run()
    check(p)


def test_captured_with_grids_that_change():
    p, eager = Program(GRIDS, 700), Program(GRIDS, 700)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        p.run()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            p.run()
    for grids in (OTHERS, GRIDS, [[0, 1, 1]] * 5, OTHERS):
        for q in (p, eager):
            q.grids.copy_(torch.tensor(grids, dtype=torch.int32, device=DEV))
            q.clear()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        eager.run()
        torch.cuda.synchronize()
        for x, y in zip(p.outputs(), eager.outputs()):
            assert torch.equal(x, y)
        if any(math.prod(g) for g in grids):
            check(p)


def test_two_streams_and_two_threads_at_once():
    """Each with its own buffers; the same bits as alone."""
    alone = Program(GRIDS, 700, seed=1)
    alone.run()
    torch.cuda.synchronize()
    both = [Program(GRIDS, 700, seed=1) for _ in range(2)]
    torch.cuda.synchronize()
    failed = []

    def work(p):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    p.run()
            st.synchronize()
        except Exception as e:      # noqa: BLE001 (told to the test's own thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(p,)) for p in both]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for p in both:
        for x, y in zip(p.outputs(), alone.outputs()):
            assert torch.equal(x, y)


def test_a_captured_first_call():
    """No call of these kernels needs to run before a capture.  (Other tests of the process may have run them: the
    head dim 24 of this one has kernels of its own only in part, the capture itself is what is tested.)"""
    st = torch.cuda.Stream()
    lens, hd = [100, 30], 24
    rows = sum(lens)
    qkv = torch.randn((rows, 3 * hd), device=DEV).to(torch.bfloat16)
    starts = torch.tensor([0, 100, 130], dtype=torch.int32, device=DEV)
    o, lse = torch.zeros((rows, hd), dtype=torch.bfloat16, device=DEV), torch.zeros((1, rows), device=DEV)
    a = dlo.make_attn_packed(batch=2, heads=1, head_dim=hd, rows_q=rows, rows_k=rows, ldq=3 * hd, ldk=3 * hd, ldv=3 * hd, ldo=hd,
                             q_starts=starts.data_ptr(), k_starts=starts.data_ptr())
    ws = torch.zeros(dlo.dlo_attention_packed_fwd_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        dlo.dlo_op_attention_packed_fwd(a, qkv.data_ptr(), qkv[:, hd:].data_ptr(), qkv[:, 2 * hd:].data_ptr(), o.data_ptr(),
                                        lse.data_ptr(), ws.data_ptr(), ws.numel(), None, st.cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    for s, n in ((0, 100), (100, 30)):
        q, k, v = (qkv[s:s + n, i * hd:(i + 1) * hd].double() for i in range(3))
        want = torch.softmax(q @ k.T / math.sqrt(hd), -1) @ v
        # P and O rounded to bf16: 2^-8 (sum p |v| + |o|), sum p |v| <= max |v|
        assert float((o[s:s + n].double() - want).abs().max()) <= 2.0 ** -7 * float(v.abs().max())
