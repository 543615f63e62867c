"""The training ops in a row, as the attention half of a block uses them, with the
error that their roundings make and no more."""
import math

import pytest
import torch

from test_gpu_train import dlo, float32_by_default, stream  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,H,hd,frame", [(2, 200, 4, 64, 20), (1, 257, 4, 72, 0), (2, 300, 3, 128, 1)])
def test_gradients_through_the_attention_half_of_a_block(B, N, H, hd, frame):
    """x -> x + attention(RMSNorm(q), RMSNorm(k), v) of q | k | v = linear(affine LayerNorm(x)), and the
    gradients of x, the norms' weights and the LayerNorm's bias, against autograd in 64 bits.

    Ten roundings to bf16 lie on the longest way (h, q | k | v, the normalised q and k, P, O in D, dS, dq | dk | dv,
    their place behind RMSNorm, dh, and o).  Each is off by u = 2^-8 of its value at most and passes on with
    a factor of about one: inputs of unit variance make logits and norms of order one.  Were they all of one sign they
    would add up to 10 u; independent, to u sqrt(10 / 3) = 1.8 u in the 2-norm.  2.5 u is asked for."""
    D = H * hd
    g = torch.Generator(device="cuda").manual_seed(N)
    rnd = lambda *s, k=1.0: torch.randn(s, generator=g, device="cuda") * k                    # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)                                                       # noqa: E731
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")                   # noqa: E731
    f32, s, R = torch.float32, stream(), B * N
    x, do = rnd(B, N, D), bf(rnd(B, N, D, k=0.1))
    W, bias = bf(rnd(3 * D, D, k=D ** -0.5)), bf(rnd(3 * D, k=0.1))
    wl, bl, wq, wk = bf(1 + rnd(D, k=0.1)), bf(rnd(D, k=0.1)), bf(1 + rnd(D, k=0.1)), bf(1 + rnd(D, k=0.1))
    lens = [N] + [N - 50] * (B - 1)
    k_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    h, mean, rstd, qkv, qk, rq, rk = e(R, D), e(R, t=f32), e(R, t=f32), e(R, 3 * D), e(R, 2 * D), e(R, t=f32), e(R, t=f32)
    o, lse, err = e(B, N, D), e(B, H, N, t=f32), torch.zeros(1, dtype=torch.int32, device="cuda")
    dlo.dlo_op_layernorm_fwd(x.data_ptr(), R, D, R, None, None, 0, wl.data_ptr(), bl.data_ptr(), 1e-6, h.data_ptr(), mean.data_ptr(),
                             rstd.data_ptr(), s)
    dlo.dlo_op_gemm(h.data_ptr(), W.data_ptr(), dlo.DT_BF16, None, 0, bias.data_ptr(), R, 3 * D, D, dlo.EPI_BIAS, qkv.data_ptr(),
                    3 * D, None, 0, 1, err.data_ptr(), s)
    for c, w, r in ((0, wq, rq), (1, wk, rk)):
        dlo.dlo_op_rmsnorm_fwd(qkv[:, c * D:].data_ptr(), 3 * D, R, D, w.data_ptr(), 1e-6, qk[:, c * D:].data_ptr(), 2 * D,
                               r.data_ptr(), s)
    a = dlo.make_attn(batch=B, heads=H, head_dim=hd, nq=N, nk=N, causal_block=frame, ldq=2 * D, ldk=2 * D, ldv=3 * D, ldo=D,
                      lddq=3 * D, lddk=3 * D, lddv=3 * D, lddo=D, k_lens=k_lens.data_ptr())
    ws = torch.empty(max(dlo.dlo_attention_fwd_workspace_bytes(a), dlo.dlo_attention_bwd_workspace_bytes(a),
                         dlo.dlo_rmsnorm_bwd_workspace_bytes(R, D), dlo.dlo_layernorm_bwd_workspace_bytes(R, D, R)),
                     dtype=torch.uint8, device="cuda")
    qkv_at = (qk.data_ptr(), qk[:, D:].data_ptr(), qkv[:, 2 * D:].data_ptr())
    dlo.dlo_op_attention_fwd(a, *qkv_at, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), err.data_ptr(), s)
    dqkv, dwq, dwk, dh, dx, dwl, dbl = e(R, 3 * D), e(D, t=f32), e(D, t=f32), e(R, D), do.float(), e(D, t=f32), e(D, t=f32)
    dlo.dlo_op_attention_bwd(a, *qkv_at, o.data_ptr(), lse.data_ptr(), do.data_ptr(), dqkv.data_ptr(), dqkv[:, D:].data_ptr(),
                             dqkv[:, 2 * D:].data_ptr(), ws.data_ptr(), ws.numel(), err.data_ptr(), s)
    for c, w, r, dw in ((0, wq, rq, dwq), (1, wk, rk, dwk)):
        t = dqkv[:, c * D:]
        dlo.dlo_op_rmsnorm_bwd(t.data_ptr(), 3 * D, qkv[:, c * D:].data_ptr(), 3 * D, w.data_ptr(), r.data_ptr(), R, D,
                               t.data_ptr(), 3 * D, dw.data_ptr(), ws.data_ptr(), ws.numel(), s)
    Wt = W.T.contiguous()
    dlo.dlo_op_gemm(dqkv.data_ptr(), Wt.data_ptr(), dlo.DT_BF16, None, 0, None, R, D, 3 * D, dlo.EPI_BIAS, dh.data_ptr(), D,
                    None, 0, 1, err.data_ptr(), s)
    # dx begins as the gradient that passes by the half on the residual path
    dlo.dlo_op_layernorm_bwd(dh.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), R, D, R, None, 0, wl.data_ptr(),
                             dx.data_ptr(), dx.data_ptr(), dbl.data_ptr(), dwl.data_ptr(), 0, ws.data_ptr(), ws.numel(), s)
    torch.cuda.synchronize()
    assert int(err.item()) == 0

    X, WL, BL, WQ, WK = (t.double().requires_grad_() for t in (x, wl, bl, wq, wk))
    mu = X.mean(-1, keepdim=True)
    Y = ((X - mu) / torch.sqrt(((X - mu) ** 2).mean(-1, keepdim=True) + 1e-6) * WL + BL) @ W.double().T + bias.double()
    rms = lambda t, w: t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w              # noqa: E731
    split = lambda t: t.reshape(B, N, H, hd).transpose(1, 2)                                  # noqa: E731
    Q, K, V = split(rms(Y[..., :D], WQ)), split(rms(Y[..., D:2 * D], WK)), split(Y[..., 2 * D:])
    i = torch.arange(N, device="cuda")
    see = (i[None, :] < k_lens[:, None])[:, None, None].expand(B, 1, N, N)
    if frame:
        see = see & (i[:, None] // frame >= i[None] // frame)
    O = (torch.softmax((Q @ K.transpose(-1, -2) / math.sqrt(hd)).masked_fill(~see, -math.inf), -1) @ V).transpose(1, 2).reshape(B, N, D)
    (X + O).backward(do.double())
    for name, got, want in (("o", o, O.detach()), ("dx", dx - do.float(), X.grad - do.double()), ("dwl", dwl, WL.grad), ("dbl", dbl, BL.grad),
                            ("dwq", dwq, WQ.grad), ("dwk", dwk, WK.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 2.5 * 2.0 ** -8, f"{name}: {rel:.3e}"
