"""torch front end of the dense operators of include/s3r_view.h: the per-head norm of queries and
keys with the rotation by position, and dense attention inside segments, forward and backward.

As in api.py, every step runs in the library's kernels on the current stream, and torch provides
the memory. All tensors must be CUDA tensors of the current device.

    q [L, H, 64], k [L, Hk, 64], v [L, Hk, 64]   bf16 (the norm also takes fp32); channels contiguous,
                                                 any token and head strides that are multiples of 8
                                                 (views of one packed projection, for example)
    pos   [L] (1-D) or [L, 2] (2-D) int32        q_offs, k_offs [segments + 1] int32
    out   [L, H, 64] bf16                        lse [H, L] fp32
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .api import _ptr, _stream

_TYPES = {torch.bfloat16: _lib.S3R_TYPE_BF16, torch.float32: _lib.S3R_TYPE_F32}


def _on_device(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device "
                         f"cuda:{torch.cuda.current_device()}")


def _rows(t: torch.Tensor, name: str, shape, dtypes) -> Tuple[int, int]:
    """Check a [L, H, 64] tensor of any strides; returns its (token, head) strides."""
    if tuple(t.shape) != tuple(shape) or t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {'/'.join(str(d) for d in dtypes)} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    if t.numel() == 0:
        return 0, 0
    if t.stride(2) != 1 or t.data_ptr() % 16 or any(
            t.shape[i] > 1 and (t.stride(i) < 64 or t.stride(i) % 8) for i in (0, 1)):
        raise ValueError(f"{name}: needs contiguous channels, a 16-byte aligned start and token and "
                         f"head strides that are multiples of 8 and at least 64; got strides "
                         f"{tuple(t.stride())}")
    _on_device(t, name)
    # a dimension of one element never steps; its stride may be anything
    head = t.stride(1) if t.shape[1] > 1 else 64
    return (t.stride(0) if t.shape[0] > 1 else head * t.shape[1]), head


def _dense(t: torch.Tensor, name: str, shape, dtype) -> None:
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")
    if t.numel():
        _on_device(t, name)
        if t.data_ptr() % 16 and t.dtype != torch.int32:
            raise ValueError(f"{name}: needs a 16-byte aligned start")


def _heads(t: torch.Tensor, name: str) -> Tuple[int, int]:
    if t.dim() != 3 or t.shape[2] != 64:
        raise ValueError(f"{name}: expected [L, H, 64], got {tuple(t.shape)}")
    return t.shape[0], t.shape[1]


# ---------------------------------------------------------------------------------------------
# norm of queries and keys with the rotation
# ---------------------------------------------------------------------------------------------
@dataclass(frozen=True)
class QKNormConfig:
    """norm: "layer" (weight and bias), "rms" (weight) or "none", over each head's 64 channels.
    rope: "1d" (pairs (i, i + 32) turned by pos * base^(-i/32)), "2d" (the first half of the
    channels by the patch row, the second by its column: pairs (i, i + 16) of each half turned by
    pos * base^(-i/16)) or "none"."""

    norm: str = "layer"
    rope: str = "2d"
    base: float = 100.0
    eps: float = 1e-6

    def _params(self, L, H, Hk, dtype, grad_dtype=None, **strides) -> _lib.QKNormParams:
        if self.norm not in _lib.NORMS or self.rope not in _lib.ROPES:
            raise ValueError(f"norm {self.norm!r} / rope {self.rope!r}: expected one of "
                             f"{tuple(_lib.NORMS)} / {tuple(_lib.ROPES)}")
        p = _lib.QKNormParams(L=L, H=H, Hk=Hk, d=64, norm=_lib.NORMS[self.norm],
                              rope=_lib.ROPES[self.rope], dtype=_TYPES[dtype],
                              grad_dtype=_TYPES[grad_dtype or dtype], eps=self.eps, base=self.base)
        for n, s in strides.items():
            setattr(p, n, (ctypes.c_int64 * 2)(*s))
        return p


def view_positions(views: int, grid_h: int, grid_w: int, special: int = 0,
                   device=None) -> torch.Tensor:
    """[views * (special + grid_h * grid_w), 2] int32 positions of a multi-view sequence for the 2-D
    rotation: each view's special tokens at (0, 0), then its patches row by row at (row + 1,
    column + 1)."""
    if min(views, grid_h, grid_w) < 1 or special < 0:
        raise ValueError("views, grid_h and grid_w must be positive, special not negative")
    r = torch.arange(1, grid_h + 1, dtype=torch.int32, device=device)
    c = torch.arange(1, grid_w + 1, dtype=torch.int32, device=device)
    patches = torch.stack(torch.meshgrid(r, c, indexing="ij"), -1).reshape(-1, 2)
    view = torch.cat([patches.new_zeros((special, 2)), patches])
    return view.repeat(views, 1)


def _check_norm(cfg: QKNormConfig, q, k, pos, weights):
    L, H = _heads(q, "q")
    Lk, Hk = _heads(k, "k")
    if Lk != L or k.dtype != q.dtype:
        raise ValueError(f"q and k must have the same tokens and type, got {tuple(q.shape)} "
                         f"{q.dtype} and {tuple(k.shape)} {k.dtype}")
    if q.dtype not in _TYPES:
        raise ValueError(f"q: expected bfloat16 or float32, got {q.dtype}")
    if cfg.rope == "none":
        if pos is not None:
            raise ValueError("pos is given, but the config has no rotation")
    else:
        if pos is None:
            raise ValueError("the rotation needs pos")
        _dense(pos, "pos", (L, 2) if cfg.rope == "2d" else (L,), torch.int32)
    for n, t in weights.items():
        if t is None:
            continue
        if cfg.norm == "none" or (n.endswith("bias") and cfg.norm != "layer"):
            raise ValueError(f"{n} is given, but norm {cfg.norm!r} has none")
        _dense(t, n, (64,), torch.float32)
    return L, H, Hk


def qk_norm_rope(cfg: QKNormConfig, q: torch.Tensor, k: torch.Tensor,
                 pos: Optional[torch.Tensor] = None, *, q_weight=None, q_bias=None, k_weight=None,
                 k_bias=None, out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norm and rotation of q and k in one pass: returns (q_out, k_out) of the inputs' type, dense
    unless out = (q_out, k_out) is given (strided outputs are taken, and the inputs themselves)."""
    L, H, Hk = _check_norm(cfg, q, k, pos, dict(q_weight=q_weight, q_bias=q_bias,
                                               k_weight=k_weight, k_bias=k_bias))
    if out is None:
        out = (torch.empty((L, H, 64), dtype=q.dtype, device=q.device),
               torch.empty((L, Hk, 64), dtype=q.dtype, device=q.device))
    qo, ko = out
    p = cfg._params(L, H, Hk, q.dtype, q_stride=_rows(q, "q", (L, H, 64), (q.dtype,)),
                    k_stride=_rows(k, "k", (L, Hk, 64), (q.dtype,)),
                    qo_stride=_rows(qo, "out[0]", (L, H, 64), (q.dtype,)),
                    ko_stride=_rows(ko, "out[1]", (L, Hk, 64), (q.dtype,)))
    if L == 0 or H + Hk == 0:
        return qo, ko
    _lib.call("s3r_qk_norm_rope_fwd", ctypes.byref(p), _ptr(q), _ptr(k), _ptr(pos), _ptr(q_weight),
              _ptr(q_bias), _ptr(k_weight), _ptr(k_bias), _ptr(qo), _ptr(ko), _stream())
    return qo, ko


class QKNormGrads(NamedTuple):
    q: torch.Tensor
    k: torch.Tensor
    q_weight: Optional[torch.Tensor]  # None where the norm has none
    q_bias: Optional[torch.Tensor]
    k_weight: Optional[torch.Tensor]
    k_bias: Optional[torch.Tensor]


def qk_norm_rope_bwd(cfg: QKNormConfig, q: torch.Tensor, k: torch.Tensor,
                     pos: Optional[torch.Tensor], dq_out: torch.Tensor, dk_out: torch.Tensor, *,
                     q_weight=None, q_bias=None, k_weight=None, k_bias=None, grads=None,
                     workspace: Optional[torch.Tensor] = None) -> QKNormGrads:
    """Gradients of qk_norm_rope for the upstream dq_out, dk_out (bf16 or fp32, both the same).

    The biases' values are not needed; passing them checks them. grads: optional (dq, dk) to write
    into, of q's type, strided or not. The weights' gradients are [64] fp32."""
    L, H, Hk = _check_norm(cfg, q, k, pos, dict(q_weight=q_weight, q_bias=q_bias,
                                               k_weight=k_weight, k_bias=k_bias))
    if dq_out.dtype not in _TYPES or dk_out.dtype != dq_out.dtype:
        raise ValueError(f"dq_out and dk_out must both be bfloat16 or float32, got {dq_out.dtype} "
                         f"and {dk_out.dtype}")
    if grads is None:
        grads = (torch.empty((L, H, 64), dtype=q.dtype, device=q.device),
                 torch.empty((L, Hk, 64), dtype=q.dtype, device=q.device))
    dq, dk = grads
    p = cfg._params(L, H, Hk, q.dtype, dq_out.dtype, q_stride=_rows(q, "q", (L, H, 64), (q.dtype,)),
                    k_stride=_rows(k, "k", (L, Hk, 64), (q.dtype,)),
                    qo_stride=_rows(dq_out, "dq_out", (L, H, 64), (dq_out.dtype,)),
                    ko_stride=_rows(dk_out, "dk_out", (L, Hk, 64), (dq_out.dtype,)),
                    dq_stride=_rows(dq, "grads[0]", (L, H, 64), (q.dtype,)),
                    dk_stride=_rows(dk, "grads[1]", (L, Hk, 64), (q.dtype,)))
    dw = torch.empty((4, 64), dtype=torch.float32, device=q.device)
    if H + Hk == 0:
        dw.zero_()
    else:
        if workspace is None:
            n = int(_lib.load().s3r_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(p)))
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
        _lib.call("s3r_qk_norm_rope_bwd", ctypes.byref(p), _ptr(q), _ptr(k), _ptr(pos),
                  _ptr(q_weight), _ptr(k_weight), _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk),
                  _ptr(dw), _ptr(workspace), workspace.numel(), _stream())
    weight, bias = cfg.norm != "none", cfg.norm == "layer"
    return QKNormGrads(dq, dk, dw[0] if weight else None, dw[1] if bias else None,
                       dw[2] if weight else None, dw[3] if bias else None)


def _as_rows(g: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    """An upstream gradient in a type and layout the backward calls take (copied only if it has to
    be: a broadcast or permuted one)."""
    if g is None:
        return torch.zeros(like.shape, dtype=like.dtype, device=like.device)
    if g.dtype not in _TYPES:
        g = g.to(like.dtype)
    return g.contiguous()


class QKNormRopeFunction(torch.autograd.Function):
    """autograd wrapper of qk_norm_rope / qk_norm_rope_bwd: apply(q, k, pos, q_weight, q_bias,
    k_weight, k_bias, cfg) -> (q_out, k_out). Saves q and k; the statistics are recomputed."""

    @staticmethod
    def forward(ctx, q, k, pos, q_weight, q_bias, k_weight, k_bias, cfg: QKNormConfig):
        ctx.cfg = cfg
        ctx.save_for_backward(q, k, pos, q_weight, q_bias, k_weight, k_bias)
        return qk_norm_rope(cfg, q, k, pos, q_weight=q_weight, q_bias=q_bias, k_weight=k_weight,
                            k_bias=k_bias)

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, pos, qw, qb, kw, kb = ctx.saved_tensors
        dq_out, dk_out = _as_rows(dq_out, q), _as_rows(dk_out, k)
        if dq_out.dtype != dk_out.dtype:
            dq_out, dk_out = dq_out.float(), dk_out.float()
        g = qk_norm_rope_bwd(ctx.cfg, q, k, pos, dq_out, dk_out, q_weight=qw, q_bias=qb,
                             k_weight=kw, k_bias=kb)
        given = (None if w is None else d for w, d in
                 ((qw, g.q_weight), (qb, g.q_bias), (kw, g.k_weight), (kb, g.k_bias)))
        return (g.q, g.k, None, *given, None)


# ---------------------------------------------------------------------------------------------
# dense attention inside segments
# ---------------------------------------------------------------------------------------------
@dataclass(frozen=True)
class ViewConfig:
    """H query heads, Hkv key/value heads (None: H; a divisor of H), and bounds on the queries and
    keys of one segment: max_q, max_k (None: every row of the tensors). Tight bounds keep the launch
    small; a segment beyond its bound is an error on the device (S3R_DEV_BAD_INDEX)."""

    H: int
    Hkv: Optional[int] = None
    max_q: Optional[int] = None
    max_k: Optional[int] = None
    scale: Optional[float] = None  # None -> 1/sqrt(64)
    test_timeout: bool = False     # testing only: exercise the bounded-wait timeout path

    @property
    def kv_heads(self) -> int:
        return self.H if self.Hkv is None else self.Hkv

    def _params(self, Lq, Lk, nseg, zero_tail, dev_status, **strides) -> _lib.ViewParams:
        p = _lib.ViewParams(Lq=Lq, Lk=Lk, H=self.H, Hkv=self.kv_heads, d=64, nseg=nseg,
                            max_q=Lq if self.max_q is None else self.max_q,
                            max_k=Lk if self.max_k is None else self.max_k,
                            scale=0.0 if self.scale is None else float(self.scale),
                            flags=(_lib.S3R_FLAG_TEST_TIMEOUT if self.test_timeout else 0)
                            | (_lib.S3R_FLAG_ZERO_TAIL if zero_tail else 0),
                            dev_status=None if dev_status is None else dev_status.data_ptr())
        for n, s in strides.items():
            setattr(p, n, (ctypes.c_int64 * 2)(*s))
        return p


def _check_view(cfg: ViewConfig, q, k, v, q_offs, k_offs):
    Lq, H = _heads(q, "q")
    Lk, Hkv = _heads(k, "k")
    if H != cfg.H or Hkv != cfg.kv_heads:
        raise ValueError(f"expected {cfg.H} query and {cfg.kv_heads} key heads, got {H} and {Hkv}")
    bf = (torch.bfloat16,)
    strides = dict(q_stride=_rows(q, "q", (Lq, H, 64), bf), k_stride=_rows(k, "k", (Lk, Hkv, 64), bf),
                   v_stride=_rows(v, "v", (Lk, Hkv, 64), bf))
    if q_offs.dim() != 1 or q_offs.numel() < 2:
        raise ValueError(f"q_offs: expected [segments + 1], got {tuple(q_offs.shape)}")
    for n, t in (("q_offs", q_offs), ("k_offs", k_offs)):
        _dense(t, n, q_offs.shape, torch.int32)
    return Lq, Lk, q_offs.numel() - 1, strides


def _workspace(fn: str, p, workspace, device) -> torch.Tensor:
    if workspace is not None:
        return workspace
    n = int(getattr(_lib.load(), fn)(ctypes.byref(p)))
    return torch.empty(n, dtype=torch.uint8, device=device)


def view_attn_fwd(cfg: ViewConfig, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  q_offs: torch.Tensor, k_offs: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense attention of each segment's queries over its own keys: returns (out [Lq, H, 64] bf16,
    lse [H, Lq] fp32). Queries without keys get 0 and -inf. Rows past the last segment are left as
    they were in an out or lse that is passed in, and are 0 and -inf in one that is allocated."""
    Lq, Lk, nseg, strides = _check_view(cfg, q, k, v, q_offs, k_offs)
    if (out is None) != (lse is None):
        raise ValueError("pass both out and lse, or neither")
    zero_tail = out is None
    if out is None:
        out = torch.empty((Lq, cfg.H, 64), dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((cfg.H, Lq), dtype=torch.float32, device=q.device)
    _dense(out, "out", (Lq, cfg.H, 64), torch.bfloat16)
    _dense(lse, "lse", (cfg.H, Lq), torch.float32)
    p = cfg._params(Lq, Lk, nseg, zero_tail, dev_status, **strides)
    ws = _workspace("s3r_view_attn_workspace_bytes", p, workspace, q.device)
    _lib.call("s3r_view_attn_fwd", ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(q_offs),
              _ptr(k_offs), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream())
    return out, lse


def view_attn_bwd(cfg: ViewConfig, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  q_offs: torch.Tensor, k_offs: torch.Tensor, out: torch.Tensor,
                  lse: torch.Tensor, dout: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, grads=None,
                  dev_status: Optional[torch.Tensor] = None):
    """Gradients of view_attn_fwd from its inputs, out and lse: returns dq, dk, dv (bf16).

    grads: optional (dq, dk, dv) to write into, strided or not; rows past the last segment are left
    as they were there, and zero in gradients allocated here."""
    Lq, Lk, nseg, strides = _check_view(cfg, q, k, v, q_offs, k_offs)
    _dense(out, "out", (Lq, cfg.H, 64), torch.bfloat16)
    _dense(lse, "lse", (cfg.H, Lq), torch.float32)
    _dense(dout, "dout", (Lq, cfg.H, 64), torch.bfloat16)
    zero_tail = grads is None
    if grads is None:
        grads = tuple(torch.empty(t.shape, dtype=torch.bfloat16, device=q.device) for t in (q, k, v))
    dq, dk, dv = grads
    for n, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        strides[n + "_stride"] = _rows(t, n, like.shape, (torch.bfloat16,))
    p = cfg._params(Lq, Lk, nseg, zero_tail, dev_status, **strides)
    ws = _workspace("s3r_view_attn_bwd_workspace_bytes", p, workspace, q.device)
    _lib.call("s3r_view_attn_bwd", ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(q_offs),
              _ptr(k_offs), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
              ws.numel(), _stream())
    return dq, dk, dv


class ViewAttentionFunction(torch.autograd.Function):
    """autograd wrapper of view_attn_fwd / view_attn_bwd: apply(q, k, v, q_offs, k_offs, cfg) -> out.
    Saves q, k, v, out and lse. The probabilities are recomputed in the backward.

    To capture a training step into a CUDA graph, capture the functional calls, or leave no eager
    autograd graph of the same leaves alive: torch's gradient accumulation would otherwise run on
    the stream of that older graph, which a capture does not allow."""

    @staticmethod
    def forward(ctx, q, k, v, q_offs, k_offs, cfg: ViewConfig):
        out, lse = view_attn_fwd(cfg, q, k, v, q_offs, k_offs)
        ctx.cfg = cfg
        ctx.save_for_backward(q, k, v, q_offs, k_offs, out, lse)
        return out

    @staticmethod
    def backward(ctx, dout):
        dout = dout.to(torch.bfloat16).contiguous()
        return (*view_attn_bwd(ctx.cfg, *ctx.saved_tensors, dout), None, None, None)
