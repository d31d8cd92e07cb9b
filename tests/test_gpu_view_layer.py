"""A run of the dense operators as a layer uses them: one packed projection, the norm with rotation, and
attention inside views (or the sparse attention over all of them), forward and backward."""
import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r

import view_ref as R

pytestmark = pytest.mark.gpu

N, GH, GW, SPECIAL, H = 3, 5, 7, 2, 2  # views of 2 + 35 tokens
P = SPECIAL + GH * GW
L = N * P


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def layer(dev, seed=5):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((L, 3, H, 64), generator=g).to(torch.bfloat16).to(dev)
    w = {n: (1 + 0.2 * torch.randn(64, generator=g)).to(dev) for n in ("q_weight", "k_weight")}
    w |= {n: (0.2 * torch.randn(64, generator=g)).to(dev) for n in ("q_bias", "k_bias")}
    dout = torch.randn((L, H, 64), generator=g).to(torch.bfloat16).to(dev)
    pos = s3r.view_positions(N, GH, GW, SPECIAL, dev)
    offs = torch.arange(0, L + 1, P, dtype=torch.int32, device=dev)
    return qkv, w, dout, pos, offs


def reference(qkv, w, dout, pos, cfg):
    """fp64 autograd of the layer, q and k rounded to bf16 between the operators like the kernels'."""
    x = qkv.double().requires_grad_()
    ws = {n: t.double().requires_grad_() for n, t in w.items()}

    def norm(t, wt, b):
        t = t - t.mean(-1, keepdim=True)
        y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + cfg.eps) * wt + b
        return R.turn(y, pos, cfg.rope, cfg.base)

    def rounded(t):  # the rounding passes the gradient
        return t + (t.to(torch.bfloat16).double() - t).detach()

    q = rounded(norm(x[:, 0], ws["q_weight"], ws["q_bias"]))
    k = rounded(norm(x[:, 1], ws["k_weight"], ws["k_bias"]))
    outs = []
    for i in range(N):
        s = slice(i * P, (i + 1) * P)
        p = torch.softmax(torch.einsum("qhc,khc->hqk", q[s], k[s]) / 8, -1)
        outs.append(torch.einsum("hqk,khc->qhc", p, x[s, 2]))
    out = torch.cat(outs)
    out.backward(dout.double())
    return out.detach(), x.grad, {n: t.grad for n, t in ws.items()}


def close(name, got, want, steps):
    """Within `steps` half steps of bf16 (2^-8 each) in the 2-norm: each operator rounds its operands and
    its results that often on the way."""
    got, want = got.double(), want.double()
    rel = ((got - want).norm() / want.norm()).item()
    assert rel <= steps * R.BF, f"{name}: {rel:.3e}"


def test_view_layer_functional_calls(dev):
    """No copies between the operators: strided projections in, gradients into one packed buffer."""
    qkv, w, dout, pos, offs = layer(dev)
    ncfg, vcfg = s3r.QKNormConfig(), s3r.ViewConfig(H=H, max_q=P, max_k=P)
    q, k = s3r.qk_norm_rope(ncfg, qkv[:, 0], qkv[:, 1], pos, **w)
    out, lse = s3r.view_attn_fwd(vcfg, q, k, qkv[:, 2], offs, offs)
    dqkv = torch.empty_like(qkv)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    s3r.view_attn_bwd(vcfg, q, k, qkv[:, 2], offs, offs, out, lse, dout, grads=(dq, dk, dqkv[:, 2]))
    g = s3r.qk_norm_rope_bwd(ncfg, qkv[:, 0], qkv[:, 1], pos, dq, dk, **w,
                             grads=(dqkv[:, 0], dqkv[:, 1]))
    want, dx, dw = reference(qkv, w, dout, pos, ncfg)
    close("out", out, want, 2)
    # P (or dS), the operator's result, the norm's result
    close("dqkv", dqkv, dx, 3)
    for n in w:
        close(n, getattr(g, n), dw[n], 3)
    # in place: the norm over its own input, the gradient over the upstream one
    buf = qkv.clone()
    q2, k2 = s3r.qk_norm_rope(ncfg, buf[:, 0], buf[:, 1], pos, **w, out=(buf[:, 0], buf[:, 1]))
    assert torch.equal(q2, q) and torch.equal(k2, k) and torch.equal(buf[:, 2], qkv[:, 2])
    g2 = s3r.qk_norm_rope_bwd(ncfg, qkv[:, 0], qkv[:, 1], pos, dq, dk, **w, grads=(dq, dk))
    assert torch.equal(g2.q, dqkv[:, 0]) and torch.equal(g2.k, dqkv[:, 1])


def test_view_layer_autograd(dev):
    qkv, w, dout, pos, offs = layer(dev)
    x = qkv.clone().requires_grad_()
    ws = {n: t.clone().requires_grad_() for n, t in w.items()}
    ncfg, vcfg = s3r.QKNormConfig(), s3r.ViewConfig(H=H, max_q=P, max_k=P)
    q, k = s3r.QKNormRopeFunction.apply(x[:, 0], x[:, 1], pos, ws["q_weight"], ws["q_bias"],
                                        ws["k_weight"], ws["k_bias"], ncfg)
    out = s3r.ViewAttentionFunction.apply(q, k, x[:, 2], offs, offs, vcfg)
    (out * dout).sum().backward()  # an upstream gradient that autograd forms
    want, dx, dw = reference(qkv, w, dout, pos, ncfg)
    close("out", out.detach(), want, 2)
    close("dqkv", x.grad, dx, 3)
    for n in w:
        close(n, ws[n].grad, dw[n], 3)
    # a broadcast upstream gradient, and an operator whose second output is not used
    x.grad = None
    q, k = s3r.QKNormRopeFunction.apply(x[:, 0], x[:, 1], pos, *(t.detach() for t in
                                        (ws["q_weight"], ws["q_bias"], ws["k_weight"], ws["k_bias"])), ncfg)
    q.float().sum().backward()
    assert torch.isfinite(x.grad).all() and (x.grad[:, 1:] == 0).all()


def test_norm_feeds_the_sparse_attention_and_takes_its_gradients(dev):
    """The global layer: the norm's outputs are what SparseAttentionFunction takes, and its fp32
    gradients (sparse_attn_bwd) go straight into qk_norm_rope_bwd."""
    qkv, w, dout, pos, _ = layer(dev, 6)
    ncfg = s3r.QKNormConfig()
    cfg = s3r.Config(L=L, H=H, block=32, topk=2)
    gates = torch.randn((L, H, 2), generator=torch.Generator().manual_seed(1)).to(dev)
    v = qkv[:, 2].contiguous()
    q, k = s3r.qk_norm_rope(ncfg, qkv[:, 0], qkv[:, 1], pos, **w)
    idx = torch.empty((H, cfg.nqb, cfg.nsel), dtype=torch.int32, device=dev)
    s3r.sparse_attn_fwd(cfg, q, k, v, gates, idx_out=idx)
    dq, dk, _, _ = s3r.sparse_attn_bwd(cfg, q, k, v, gates, idx, dout)
    assert dq.dtype == torch.float32
    g = s3r.qk_norm_rope_bwd(ncfg, qkv[:, 0], qkv[:, 1], pos, dq, dk, **w)
    for n, x, up in (("q", qkv[:, 0], dq), ("k", qkv[:, 1], dk)):
        dx, dw, db = R.qk_norm_rope_bwd(x, pos, w[n + "_weight"], up, "layer", "2d", ncfg.base, ncfg.eps)
        close("d" + n, getattr(g, n), dx, 1)
        torch.testing.assert_close(getattr(g, n + "_weight").double(), dw, rtol=1e-4, atol=1e-4)
        torch.testing.assert_close(getattr(g, n + "_bias").double(), db, rtol=1e-4, atol=1e-4)


def test_dense_attention_is_the_sparse_one_with_every_block(dev):
    """Every block selected and the compression gate shut: the sparse path is dense attention, and so
    is view_attn over one segment."""
    qkv, w, dout, pos, _ = layer(dev, 7)
    q, k, v = (qkv[:, i].contiguous() for i in range(3))
    cfg = s3r.Config(L=L, H=H, block=32, topk=-(-L // 32))
    gates = torch.full((L, H, 2), 1e4, device=dev)
    gates[..., 0] = -1e4
    sparse = s3r.sparse_attn_fwd(cfg, q, k, v, gates)
    offs = torch.tensor([0, L], dtype=torch.int32, device=dev)
    dense, _ = s3r.view_attn_fwd(s3r.ViewConfig(H=H), q, k, v, offs, offs)
    close("dense", dense, sparse, 3)


@pytest.mark.parametrize("H_,L_", [(16, 2_200_000)])
def test_norm_beyond_32_bit_element_offsets(dev, H_, L_):
    g = torch.Generator(device=dev).manual_seed(8)
    x = torch.randn((L_, H_, 64), generator=g, device=dev, dtype=torch.bfloat16)
    pos = torch.arange(L_, dtype=torch.int32, device=dev)
    cfg = s3r.QKNormConfig(norm="rms", rope="1d", base=1e4)
    y, _ = s3r.qk_norm_rope(cfg, x, x[:, :1], pos)
    for s in (slice(0, 50), slice(L_ - 50, L_)):
        want = R.qk_norm_rope(x[s], pos[s], None, None, "rms", "1d", 1e4, cfg.eps)
        assert ((y[s].double() - want).abs() <= R.BF * want.abs() + 1e-5).all()
    gr = s3r.qk_norm_rope_bwd(cfg, x, x[:, :1], pos, y, y[:, :1])
    s = slice(L_ - 50, L_)
    dx, _, _ = R.qk_norm_rope_bwd(x[s], pos[s], None, y[s], "rms", "1d", 1e4, cfg.eps)
    # dx is a difference of terms of order 1 that nearly cancel (the gradient of a row's own direction)
    assert ((gr.q[s].double() - dx).abs() <= R.BF * dx.abs() + 1e-4).all()


def test_autograd_takes_any_upstream_gradient(dev):
    """Gradients that start inside 16 bytes or are broadcast, and no second derivative."""
    g = torch.Generator(device=dev).manual_seed(9)
    t = [torch.randn((40, 2, 64), generator=g, device=dev).to(torch.bfloat16).requires_grad_() for _ in range(3)]
    o = torch.tensor([0, 40], dtype=torch.int32, device=dev)
    one, c = torch.ones(1, dtype=torch.bfloat16, device=dev), s3r.QKNormConfig(norm="rms", rope="none")
    up = torch.randn(5121, generator=g, device=dev).to(torch.bfloat16)
    attend = lambda q, k, v: s3r.ViewAttentionFunction.apply(q, k, v, o, o, s3r.ViewConfig(H=2))
    norm = lambda q, k, v: s3r.QKNormRopeFunction.apply(q, k, None, None, None, None, None, c)[0]
    for f, n in ((attend, 3), (norm, 1)):
        want = torch.autograd.grad(f(*t), t[:n], up[1:].clone().view(40, 2, 64))
        got = torch.autograd.grad(torch.cat([one, f(*t).reshape(-1)]), t[:n], up)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        want = torch.autograd.grad(f(*t), t[:n], torch.ones((40, 2, 64), dtype=torch.bfloat16, device=dev))
        got = torch.autograd.grad(f(*t).sum(), t[:n], create_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        with pytest.raises(RuntimeError):
            got[0].float().pow(2).sum().backward()
