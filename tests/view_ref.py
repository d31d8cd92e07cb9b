"""Plain fp64 forms of the dense operators of include/s3r_view.h, with elementwise error bounds.

Half a rounding step of bf16 is 2^-8 of the value, of fp32 2^-24. The kernels round to bf16: P (and
dS) before a product, and each result once. A product in fp32 of n terms is off by at most about
n 2^-24 of the sum of the terms' magnitudes; the exponential by 2^-22 of its value.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

BF = 2.0 ** -8   # half a step of bf16
F32 = 2.0 ** -24


class Attn(NamedTuple):
    out: torch.Tensor      # [Lq, H, 64]
    lse: torch.Tensor      # [H, Lq]
    out_err: torch.Tensor  # bounds of the kernels' errors, same shapes
    lse_err: torch.Tensor
    dq: Optional[torch.Tensor] = None
    dk: Optional[torch.Tensor] = None
    dv: Optional[torch.Tensor] = None
    dq_err: Optional[torch.Tensor] = None
    dk_err: Optional[torch.Tensor] = None
    dv_err: Optional[torch.Tensor] = None


def attention(q, k, v, q_offs, k_offs, scale=0.125, dout=None) -> Attn:
    """q [Lq, H, 64], k, v [Lk, Hkv, 64], offsets as lists; rows of no segment give 0 / -inf."""
    q, k, v = q.double(), k.double(), v.double()
    H, group = q.shape[1], q.shape[1] // k.shape[1]
    z = lambda t: torch.zeros_like(t)  # noqa: E731
    out, out_err, dq, dq_err = z(q), z(q), z(q), z(q)
    dk, dv, dk_err, dv_err = z(k), z(k), z(k), z(k)
    lse = torch.full((H, q.shape[0]), -torch.inf, dtype=torch.float64, device=q.device)
    lse_err = torch.zeros_like(lse)
    for s in range(len(q_offs) - 1):
        a, b = slice(q_offs[s], q_offs[s + 1]), slice(k_offs[s], k_offs[s + 1])
        if a.stop <= a.start or b.stop <= b.start:
            continue
        for h in range(H):
            x, y, w = q[a, h], k[b, h // group], v[b, h // group]
            t = scale * x @ y.T
            z_ = torch.logsumexp(t, 1, keepdim=True)
            p = torch.exp(t - z_)
            # a logit is a 64-term product, a scaling and a difference to the row's reference
            slack = 70 * F32 * scale * (x.abs() @ y.abs().T) + 8 * F32 * (t.abs() + z_.abs())
            rel = slack + slack.amax(1, keepdim=True) + 2.0 ** -20  # of each P
            mass = p @ w.abs()
            out[a, h], lse[h, a] = p @ w, z_[:, 0]
            out_err[a, h] = (p * (BF + rel)) @ w.abs() + BF * out[a, h].abs() + 1e-5 * mass
            lse_err[h, a] = slack.amax(1) + 2.0 ** -20 + 4 * F32 * z_[:, 0].abs()
            if dout is None:
                continue
            go = dout[a, h].double()
            dp = go @ w.T
            d = (go * out[a, h]).sum(1, keepdim=True)
            # D comes from the bf16 out the forward wrote, or, up to 256 keys, from P and dP in fp32
            d_err = (go.abs() * out_err[a, h]).sum(1, keepdim=True)
            if p.shape[1] <= 256:
                each = 70 * F32 * (go.abs() @ w.abs().T)  # of a dP
                d_err = (p * ((rel + 256 * F32) * dp.abs() + each)).sum(1, keepdim=True)
            ds = p * (dp - d)
            ds_err = BF * ds.abs() + p * (d_err + 70 * F32 * (go.abs() @ w.abs().T)) + rel * ds.abs()
            many = 1e-5  # fp32 sums over the walk, of the terms' magnitudes
            dq[a, h] = scale * ds @ y
            dq_err[a, h] = scale * (ds_err + many * ds.abs()) @ y.abs() + BF * dq[a, h].abs()
            dk[b, h // group] += scale * ds.T @ x
            dk_err[b, h // group] += scale * (ds_err + many * ds.abs()).T @ x.abs()
            dv[b, h // group] += p.T @ go
            dv_err[b, h // group] += (p * (BF + rel + many)).T @ go.abs()
    if dout is None:
        return Attn(out, lse, out_err, lse_err)
    return Attn(out, lse, out_err, lse_err, dq, dk, dv, dq_err, dk_err + BF * dk.abs(),
                dv_err + BF * dv.abs())


def angles(pos, rope, base):
    """[L, 64] angle of each channel (a pair's two channels have the same)."""
    p, c = pos.double(), torch.arange(64, device=pos.device)
    if rope == "1d":
        return p[:, None] * base ** (-(c % 32).double() / 32)
    return p[:, (c >= 32).long()] * base ** (-(c % 16).double() / 16)


def turn(y, pos, rope, base, back=False):
    """R y (or R^T y) for y [L, H, 64]."""
    if rope == "none":
        return y
    a = angles(pos, rope, base)[:, None]
    c = torch.arange(64, device=y.device)
    partner, first = (c ^ 32, c < 32) if rope == "1d" else (c ^ 16, (c & 16) == 0)
    sign = torch.where(first, -1.0, 1.0).double() * (-1 if back else 1)
    return y * a.cos() + y[..., partner] * a.sin() * sign


def normed(x, norm, eps):
    """(xhat, 1 / sigma)"""
    x = x.double()
    if norm == "none":
        return x, torch.ones_like(x[..., :1])
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, r


def qk_norm_rope(x, pos, w, b, norm, rope, base, eps):
    y = normed(x, norm, eps)[0]
    y = y * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return turn(y, pos, rope, base)


def qk_norm_rope_bwd(x, pos, w, g, norm, rope, base, eps):
    """dx, dweight, dbias"""
    xhat, r = normed(x, norm, eps)
    dy = turn(g.double(), pos, rope, base, back=True)
    h = dy * (1.0 if w is None else w.double())
    dx = h
    if norm != "none":
        dx = h - xhat * (h * xhat).mean(-1, keepdim=True)
    if norm == "layer":
        dx = dx - h.mean(-1, keepdim=True)
    return dx * r, (dy * xhat).sum((0, 1)), dy.sum((0, 1))
