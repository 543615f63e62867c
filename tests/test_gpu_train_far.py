"""Training ops where offsets pass 32 bits, where the first call of a process is
captured, and where two host threads call at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from test_gpu_train import NORM_F, U, Problem, dlo, float32_by_default, ptr, stream, within  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("nq,cb,lens", [(70, 0, None), (70, 1, [70, 33, 70])], ids=["full", "causal-lens"])
def test_attention_rows_far_apart(nq, cb, lens):
    """Rows 2^24 elements apart in one buffer of 3.5e9: the third sequence lies behind 2^31."""
    B, H, G, hd, ld = 3, 4, 2, 64, 1 << 24
    near = Problem(B, H, G, hd, nq, nq, cb, lens, lens, seed=41, fused=False)
    far = Problem(B, H, G, hd, nq, nq, cb, lens, lens, seed=41, fused=False)
    rows = torch.empty((B, nq, ld), dtype=torch.bfloat16, device="cuda")
    at = 0

    def place(t):
        nonlocal at
        view = rows[..., at:at + t.shape[-1]]
        view.copy_(t)
        at += t.shape[-1] + 64
        return view

    for n in ("q", "k", "v", "do", "o"):
        setattr(far, n, place(getattr(far, n)))
    got = [place(t) for t in far.grads()]
    want = near.grads()
    for p, g in ((near, want), (far, got)):
        p.forward()
        p.backward(g)
    torch.cuda.synchronize()
    assert int(near.err.item()) == 0 and int(far.err.item()) == 0
    for a, b in zip((near.o, near.lse, *want), (far.o, far.lse, *got)):
        assert torch.equal(a, b)


def test_layernorm_of_more_than_2_to_the_31_elements():
    rows, D, rpb = 430080, 5120, 215040
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((rows, D), generator=g, device="cuda")
    dy = torch.randn((rows, D), generator=g, device="cuda").to(torch.bfloat16)
    mod = torch.randn((2, 2 * D), generator=g, device="cuda") * 0.3
    y, mean, rstd = torch.empty_like(dy), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dlo.dlo_op_layernorm_fwd(ptr(x), rows, D, rpb, ptr(mod), ptr(mod[:, D:]), 2 * D, None, None, 1e-6, ptr(y), ptr(mean), ptr(rstd), stream())
    dx, dmod = torch.empty_like(x), torch.empty_like(mod)
    ws = torch.empty(dlo.dlo_layernorm_bwd_workspace_bytes(rows, D, rpb), dtype=torch.uint8, device="cuda")
    dlo.dlo_op_layernorm_bwd(ptr(dy), ptr(x), ptr(mean), ptr(rstd), rows, D, rpb, ptr(mod[:, D:]), 2 * D, None, None, ptr(dx), ptr(dmod),
                             ptr(dmod[:, D:]), 2 * D, ptr(ws), ws.numel(), stream())
    torch.cuda.synchronize()
    far = slice(rows - 200, rows)                    # all of it behind 2^31 elements
    X, DY, gain, add = x[far].double(), dy[far].double(), 1 + mod[1, D:].double(), mod[1, :D].double()
    mu = X.mean(1, keepdim=True)
    rs = 1 / torch.sqrt(((X - mu) ** 2).mean(1, keepdim=True) + 1e-6)
    xh, gg = (X - mu) * rs, DY * gain
    span = X.abs().amax(1, keepdim=True) * rs
    within(y[far], xh * gain + add, U * (xh * gain + add).abs() + NORM_F * ((span + 1) * gain.abs() + add.abs()) + 1e-30, "y")
    want = rs * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    size = rs * (gg.abs() + gg.abs().mean(1, keepdim=True) + (xh.abs() + 1) * (gg * xh).abs().mean(1, keepdim=True))
    within(dx[far], want, NORM_F * (1 + span) * size + 1e-30, "dx")
    # sums over 215040 rows: chains of about 1415 rows a CTA, each addition off by 2^-24 of the chain's sum of magnitudes
    for b in range(2):
        s1, s2, b1, b2 = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(4))
        for i in range(b * rpb, (b + 1) * rpb, 8192):
            r = slice(i, min(i + 8192, (b + 1) * rpb))
            d, h = dy[r].double(), (x[r].double() - mean[r].double()[:, None]) * rstd[r].double()[:, None]
            s1, s2, b1, b2 = s1 + d.sum(0), s2 + (d * h).sum(0), b1 + d.abs().sum(0), b2 + (d * h).abs().sum(0)
        within(dmod[b, :D], s1, 1500 * 2.0 ** -24 * b1, "dshift")
        within(dmod[b, D:], s2, 1500 * 2.0 ** -24 * b2, "dscale")


def test_rmsnorm_rows_far_apart():
    rows, D, ld = 200, 1152, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(4)
    near = [torch.randn((rows, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    w = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    big = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    far = [big[:, i * 2048:i * 2048 + D] for i in range(4)]
    far[0].copy_(near[0])
    far[1].copy_(near[1])
    out = []
    for x, dy, y, dx in ((*near, torch.empty_like(near[0]), torch.empty_like(near[0])), far):
        l = x.stride(0)
        rstd, dw = torch.empty(rows, device="cuda"), torch.empty(D, device="cuda")
        ws = torch.empty(dlo.dlo_rmsnorm_bwd_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
        dlo.dlo_op_rmsnorm_fwd(ptr(x), l, rows, D, ptr(w), 1e-6, ptr(y), l, ptr(rstd), stream())
        dlo.dlo_op_rmsnorm_bwd(ptr(dy), l, ptr(x), l, ptr(w), ptr(rstd), rows, D, ptr(dx), l, ptr(dw), ptr(ws), ws.numel(), stream())
        out.append((y, dx, rstd, dw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*out)) and torch.isfinite(out[0][1]).all()


FIRST = """
import sys
sys.path[:0] = ["tests", "."]
import torch
from test_gpu_train import Problem, dlo, ptr, stream
p = Problem(2, 4, 2, 72, 300, 300, 50, [300, 190], [280, 300])
q = Problem(1, 2, 1, 64, 5, 4100)             # its keys are split
grads, gq = p.grads(), q.grads()
rows, D = 300, 1152
x = torch.randn((rows, D), device="cuda")
dy, w = torch.randn((rows, D), device="cuda").to(torch.bfloat16), torch.ones(D, dtype=torch.bfloat16, device="cuda")
y, xb, dxb, dx = torch.empty_like(dy), x.to(torch.bfloat16), torch.empty_like(dy), torch.empty_like(x)
mean, rstd, a, b = (torch.empty(n, device="cuda") for n in (rows, rows, D, D))
def size(f, r): return torch.empty(f(r), dtype=torch.uint8, device="cuda")
wp = size(dlo.dlo_attention_fwd_workspace_bytes, p.desc()), size(dlo.dlo_attention_bwd_workspace_bytes, p.desc(grads))
wq = size(dlo.dlo_attention_fwd_workspace_bytes, q.desc()), size(dlo.dlo_attention_bwd_workspace_bytes, q.desc(gq))
ws = torch.empty(max(dlo.dlo_layernorm_bwd_workspace_bytes(rows, D, rows), dlo.dlo_rmsnorm_bwd_workspace_bytes(rows, D)), dtype=torch.uint8, device="cuda")
def norms():
    s = stream()
    dlo.dlo_op_layernorm_fwd(ptr(x), rows, D, rows, None, None, 0, ptr(w), ptr(w), 1e-6, ptr(y), ptr(mean), ptr(rstd), s)
    dlo.dlo_op_layernorm_bwd(ptr(dy), ptr(x), ptr(mean), ptr(rstd), rows, D, rows, None, 0, ptr(w), None, ptr(dx), ptr(a), ptr(b), 0, ptr(ws), ws.numel(), s)
    dlo.dlo_op_rmsnorm_fwd(ptr(xb), D, rows, D, ptr(w), 1e-6, ptr(y), D, ptr(rstd), s)
    dlo.dlo_op_rmsnorm_bwd(ptr(dy), D, ptr(xb), D, ptr(w), ptr(rstd), rows, D, ptr(dxb), D, ptr(b), ptr(ws), ws.numel(), s)
def everything():
    p.forward(wp[0]); p.backward(grads, wp[1]); q.forward(wq[0]); q.backward(gq, wq[1]); norms()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    everything()
outs = [p.o, p.lse, q.o, q.lse, *grads, *gq, y, dx, dxb, a, b, rstd]
for t in outs: t.fill_(7.0)
g.replay()
torch.cuda.synchronize()
keep = [t.clone() for t in outs]
everything()
torch.cuda.synchronize()
assert all(torch.equal(torch.nan_to_num(s), torch.nan_to_num(t)) for s, t in zip(keep, outs))
p.check(p.reference(), grads)
q.check(q.reference(), gq)
print("same")
"""


def test_the_first_call_of_a_process_may_be_a_captured_one():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_two_host_threads_call_at_once():
    problems = [Problem(2, 4, 2, 64, 300, 300, 50, [300, 190], [280, 300], seed=70 + i) for i in range(2)]
    want = []
    for p in problems:
        p.forward()
        want.append(p.grads())
        p.backward(want[-1])
    torch.cuda.synchronize()
    o = [p.o.clone() for p in problems]
    failed, begin = [], threading.Barrier(2)

    def work(i):
        try:
            p, side = problems[i], torch.cuda.Stream()
            with torch.cuda.stream(side):
                grads = p.grads()
                wf, wb = p.forward(), p.backward(grads)
                side.synchronize()
                begin.wait(60)
                for _ in range(200):
                    p.forward(wf)
                    p.backward(grads, wb)
                side.synchronize()
                assert int(p.err.item()) == 0 and torch.equal(p.o, o[i])
                assert all(torch.equal(a, b) for a, b in zip(grads, want[i]))
        except BaseException as e:      # noqa: BLE001 -- carried to the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]
