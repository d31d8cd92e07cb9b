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
from torch.autograd.function import once_differentiable

from . import _lib

_TYPES = {torch.bfloat16: _lib.S3R_TYPE_BF16, torch.float32: _lib.S3R_TYPE_F32}
_BF16 = (torch.bfloat16,)
_C = torch._C


# Small calls are bound by this file: the stream's handle without an object, and the current device of
# a process that has a CUDA tensor. Looked up in the call: a torch built without CUDA has neither, and
# the package can be imported there.
def _raw_stream(device: int) -> int:
    return _C._cuda_getCurrentRawStream(device)


def _current_device() -> int:
    return _C._cuda_getDevice()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _device(t: torch.Tensor) -> int:
    """The call's device: the current one, which t has to be on."""
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    d = _current_device()
    if t.get_device() != d:
        raise ValueError(f"a tensor is on {t.device}, not on the current device cuda:{d}")
    return d


def _wrong_device(t: torch.Tensor, name: str, device: int) -> ValueError:
    return ValueError(f"{name} is on {t.device}, not on the current device cuda:{device}")


def _new(t: torch.Tensor, shape) -> torch.Tensor:
    """A dense tensor of t's type and device (the quicker call where t has the shape and is dense)."""
    return torch.empty_like(t) if t.shape == shape and t.is_contiguous() else t.new_empty(shape)


def _rows(t: torch.Tensor, name: str, shape, dtypes, device: int) -> Tuple[int, int]:
    """Check a [L, H, 64] tensor of any strides; returns its (token, head) strides."""
    L, H, _ = shape
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {'/'.join(str(d) for d in dtypes)} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    if t.get_device() != device:
        raise _wrong_device(t, name, device)
    if L == 0 or H == 0:
        return 0, 0
    tok, head, channel = t.stride()
    # a dimension of one element never steps; its stride may be anything
    if H == 1:
        head = 64
    if L == 1:
        tok = head * H
    if channel != 1 or t.data_ptr() % 16 or tok < 64 or head < 64 or tok % 8 or head % 8:
        raise ValueError(f"{name}: needs contiguous channels, a 16-byte aligned start and token and "
                         f"head strides that are multiples of 8 and at least 64; got strides "
                         f"{tuple(t.stride())}")
    return tok, head


def _dense(t: torch.Tensor, name: str, shape, dtype, device: int) -> None:
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")
    if t.get_device() != device:
        raise _wrong_device(t, name, device)
    if dtype is not torch.int32 and t.data_ptr() % 16:
        raise ValueError(f"{name}: needs a 16-byte aligned start")


def _workspace(t: Optional[torch.Tensor], n: int, like: torch.Tensor,
               device: int) -> Optional[torch.Tensor]:
    """A call's workspace: t, checked to hold n bytes, or n bytes allocated (None for none)."""
    if t is None:
        return like.new_empty(n, dtype=torch.uint8) if n else None
    if t.get_device() != device:
        raise _wrong_device(t, "workspace", device)
    if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < n or t.data_ptr() % 256:
        raise ValueError(f"workspace: expected {n} contiguous bytes (uint8), 256-byte aligned; got "
                         f"{t.dtype} {tuple(t.shape)}")
    return t


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

    def _params(self, L, H, Hk, dtype, grad_dtype, q, k, qo, ko, dq=(0, 0),
                dk=(0, 0)) -> _lib.QKNormParams:
        return _lib.QKNormParams(L, H, Hk, 64, _lib.NORMS[self.norm], _lib.ROPES[self.rope],
                                 _TYPES[dtype], _TYPES[grad_dtype], self.eps, self.base, *q, *k, *qo,
                                 *ko, *dq, *dk)


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


def _check_norm(cfg: QKNormConfig, q, k, pos, q_weight, q_bias, k_weight, k_bias):
    if cfg.norm not in _lib.NORMS or cfg.rope not in _lib.ROPES:
        raise ValueError(f"norm {cfg.norm!r} / rope {cfg.rope!r}: expected one of "
                         f"{tuple(_lib.NORMS)} / {tuple(_lib.ROPES)}")
    L, H = _heads(q, "q")
    Lk, Hk = _heads(k, "k")
    if Lk != L or k.dtype != q.dtype or q.dtype not in _TYPES:
        raise ValueError(f"q and k must have the same tokens and type, bfloat16 or float32; got "
                         f"{tuple(q.shape)} {q.dtype} and {tuple(k.shape)} {k.dtype}")
    device = _device(q)
    if cfg.rope == "none":
        if pos is not None:
            raise ValueError("pos is given, but the config has no rotation")
    elif pos is None:
        raise ValueError("the rotation needs pos")
    else:
        _dense(pos, "pos", (L, 2) if cfg.rope == "2d" else (L,), torch.int32, device)
    for n, t in (("q_weight", q_weight), ("k_weight", k_weight), ("q_bias", q_bias), ("k_bias", k_bias)):
        if t is not None:
            if cfg.norm == "none" or (n[2:] == "bias" and cfg.norm != "layer"):
                raise ValueError(f"{n} is given, but norm {cfg.norm!r} has none")
            _dense(t, n, (64,), torch.float32, device)
    return L, H, Hk, device


def qk_norm_rope(cfg: QKNormConfig, q: torch.Tensor, k: torch.Tensor,
                 pos: Optional[torch.Tensor] = None, *, q_weight=None, q_bias=None, k_weight=None,
                 k_bias=None, out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norm and rotation of q and k in one pass: returns (q_out, k_out) of the inputs' type, dense
    unless out = (q_out, k_out) is given (strided outputs are taken, and the inputs themselves, each in
    its own place; no other overlap)."""
    L, H, Hk, device = _check_norm(cfg, q, k, pos, q_weight, q_bias, k_weight, k_bias)
    dtype = (q.dtype,)
    qs, ks = _rows(q, "q", (L, H, 64), dtype, device), _rows(k, "k", (L, Hk, 64), dtype, device)
    if out is None:
        qo, ko = _new(q, (L, H, 64)), _new(k, (L, Hk, 64))
        p = cfg._params(L, H, Hk, q.dtype, q.dtype, qs, ks, (0, 0), (0, 0))
    else:
        qo, ko = out
        p = cfg._params(L, H, Hk, q.dtype, q.dtype, qs, ks,
                        _rows(qo, "out[0]", (L, H, 64), dtype, device),
                        _rows(ko, "out[1]", (L, Hk, 64), dtype, device))
    if L and H + Hk:
        _lib.call("s3r_qk_norm_rope_fwd", ctypes.byref(p), q.data_ptr(), k.data_ptr(), _ptr(pos),
                  _ptr(q_weight), _ptr(q_bias), _ptr(k_weight), _ptr(k_bias), qo.data_ptr(),
                  ko.data_ptr(), _raw_stream(device))
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
    L, H, Hk, device = _check_norm(cfg, q, k, pos, q_weight, q_bias, k_weight, k_bias)
    if dq_out.dtype not in _TYPES or dk_out.dtype != dq_out.dtype:
        raise ValueError(f"dq_out and dk_out must both be bfloat16 or float32, got {dq_out.dtype} "
                         f"and {dk_out.dtype}")
    dtype, gtype, qshape, kshape = (q.dtype,), (dq_out.dtype,), (L, H, 64), (L, Hk, 64)
    strides = [_rows(q, "q", qshape, dtype, device), _rows(k, "k", kshape, dtype, device),
               _rows(dq_out, "dq_out", qshape, gtype, device),
               _rows(dk_out, "dk_out", kshape, gtype, device)]
    if grads is None:
        dq, dk = _new(q, qshape), _new(k, kshape)
    else:
        dq, dk = grads
        strides += [_rows(dq, "grads[0]", qshape, dtype, device),
                    _rows(dk, "grads[1]", kshape, dtype, device)]
    dw = q.new_empty((4, 64), dtype=torch.float32)
    if H + Hk == 0:
        dw.zero_()
    else:
        p = cfg._params(L, H, Hk, q.dtype, dq_out.dtype, *strides)
        workspace = _workspace(
            workspace, _lib.load().s3r_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(p)), q, device)
        _lib.call("s3r_qk_norm_rope_bwd", ctypes.byref(p), q.data_ptr(), k.data_ptr(), _ptr(pos),
                  _ptr(q_weight), _ptr(k_weight), dq_out.data_ptr(), dk_out.data_ptr(),
                  dq.data_ptr(), dk.data_ptr(), dw.data_ptr(), _ptr(workspace),
                  0 if workspace is None else workspace.numel(), _raw_stream(device))
    if cfg.norm == "none":
        return QKNormGrads(dq, dk, None, None, None, None)
    dqw, dqb, dkw, dkb = dw.unbind()
    return QKNormGrads(dq, dk, dqw, dqb, dkw, dkb) if cfg.norm == "layer" else \
        QKNormGrads(dq, dk, dqw, None, dkw, None)


def _as_rows(g: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    """An upstream gradient in a type and layout the backward calls take (copied only if it has to
    be: a broadcast or permuted one, or one that starts inside 16 bytes)."""
    if g is None:
        return torch.zeros(like.shape, dtype=like.dtype, device=like.device)
    if g.dtype not in _TYPES:
        g = g.to(like.dtype)
    g = g.contiguous()
    return g.clone() if g.data_ptr() % 16 else g


class QKNormRopeFunction(torch.autograd.Function):
    """autograd wrapper of qk_norm_rope / qk_norm_rope_bwd: apply(q, k, pos, q_weight, q_bias,
    k_weight, k_bias, cfg) -> (q_out, k_out). Saves q and k; the statistics are recomputed. Captured into a
    CUDA graph: as for ViewAttentionFunction."""

    @staticmethod
    def forward(ctx, q, k, pos, q_weight, q_bias, k_weight, k_bias, cfg: QKNormConfig):
        ctx.cfg = cfg
        ctx.save_for_backward(q, k, pos, q_weight, q_bias, k_weight, k_bias)
        return qk_norm_rope(cfg, q, k, pos, q_weight=q_weight, q_bias=q_bias, k_weight=k_weight,
                            k_bias=k_bias)

    @staticmethod
    @once_differentiable
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
_INT32_MAX = 2 ** 31 - 1


def _bound(most: Optional[int], rows: int) -> int:
    """The bound on a segment's rows as the library takes it: the tensor's rows bound it too; a
    negative one, which the library refuses, stays negative."""
    return rows if most is None else max(-1, min(most, rows))


@dataclass(frozen=True)
class ViewConfig:
    """H query heads, Hkv key/value heads (None: H; a divisor of H), and bounds on the queries and
    keys of one segment: max_q, max_k (None: every row of the tensors). Tight bounds keep the launch
    small (more than 2^31 blocks are refused, and each without rows takes an SM about 0.5 us); a segment
    beyond its bound is an error on the device (S3R_DEV_BAD_INDEX)."""

    H: int
    Hkv: Optional[int] = None
    max_q: Optional[int] = None
    max_k: Optional[int] = None
    scale: Optional[float] = None  # None -> 1/sqrt(64)
    test_timeout: bool = False     # testing only: exercise the bounded-wait timeout path

    @property
    def kv_heads(self) -> int:
        return self.H if self.Hkv is None else self.Hkv

    def _params(self, Lq, Lk, nseg, all_rows, dev_status, strides) -> _lib.ViewParams:
        # (what does not fit the library's fields would reach it as another value: 2^32 + 5 as 5, and a
        # scale that is 0 in fp32 as the default)
        if self.scale is not None and not 0 < ctypes.c_float(self.scale).value < float("inf"):
            raise ValueError(f"scale must be positive and finite in fp32, got {self.scale}")
        if nseg > _INT32_MAX:
            raise ValueError(f"expected at most 2^31 - 1 segments, got {nseg}")
        return _lib.ViewParams(Lq, Lk, self.H, self.kv_heads, 64, nseg,
                               _bound(self.max_q, Lq), _bound(self.max_k, Lk),
                               0.0 if self.scale is None else self.scale,
                               (_lib.S3R_FLAG_TEST_TIMEOUT if self.test_timeout else 0)
                               | (_lib.S3R_FLAG_ALL_ROWS if all_rows else 0), *strides,
                               _ptr(dev_status))


def _check_view(cfg: ViewConfig, q, k, v, q_offs, k_offs, dev_status):
    Lq, H = _heads(q, "q")
    Lk, Hkv = _heads(k, "k")
    if H != cfg.H or Hkv != cfg.kv_heads:
        raise ValueError(f"expected {cfg.H} query and {cfg.kv_heads} key heads, got {H} and {Hkv}")
    device = _device(q)
    strides = (*_rows(q, "q", (Lq, H, 64), _BF16, device), *_rows(k, "k", (Lk, Hkv, 64), _BF16, device),
               *_rows(v, "v", (Lk, Hkv, 64), _BF16, device))
    if q_offs.dim() != 1 or q_offs.shape[0] < 2:
        raise ValueError(f"q_offs: expected [segments + 1], got {tuple(q_offs.shape)}")
    _dense(q_offs, "q_offs", q_offs.shape, torch.int32, device)
    _dense(k_offs, "k_offs", q_offs.shape, torch.int32, device)
    if dev_status is not None:
        _dense(dev_status, "dev_status", (1,), torch.int32, device)
    return Lq, Lk, q_offs.shape[0] - 1, strides, device


def view_attn_fwd(cfg: ViewConfig, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  q_offs: torch.Tensor, k_offs: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense attention of each segment's queries over its own keys: returns (out [Lq, H, 64] bf16,
    lse [H, Lq] fp32). Queries without keys get 0 and -inf. Rows of no segment (before the first,
    past the last) are left as they were in an out and lse that are passed in, and are 0 and -inf in
    allocated ones.

    out and lse must not overlap the inputs. A segment whose offsets cannot be used (descending, past the
    tensors, longer than the config's bounds) is not computed: its rows are left as they were, or NaN in
    allocated results, and dev_status (one int32, read with read_device_status) says so."""
    Lq, Lk, nseg, strides, device = _check_view(cfg, q, k, v, q_offs, k_offs, dev_status)
    if (out is None) != (lse is None):
        raise ValueError("pass both out and lse, or neither")
    all_rows = out is None
    if all_rows:
        out, lse = _new(q, (Lq, cfg.H, 64)), q.new_empty((cfg.H, Lq), dtype=torch.float32)
    else:
        _dense(out, "out", (Lq, cfg.H, 64), torch.bfloat16, device)
        _dense(lse, "lse", (cfg.H, Lq), torch.float32, device)
    p = cfg._params(Lq, Lk, nseg, all_rows, dev_status, (*strides, 0, 0, 0, 0, 0, 0))
    workspace = _workspace(workspace, _lib.load().s3r_view_attn_workspace_bytes(ctypes.byref(p)), q,
                           device)
    _lib.call("s3r_view_attn_fwd", ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
              q_offs.data_ptr(), k_offs.data_ptr(), out.data_ptr(), lse.data_ptr(),
              _ptr(workspace), 0 if workspace is None else workspace.numel(), _raw_stream(device))
    return out, lse


def view_attn_bwd(cfg: ViewConfig, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  q_offs: torch.Tensor, k_offs: torch.Tensor, out: torch.Tensor,
                  lse: torch.Tensor, dout: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, grads=None,
                  dev_status: Optional[torch.Tensor] = None):
    """Gradients of view_attn_fwd from its inputs, out and lse: returns dq, dk, dv (bf16).

    grads: optional (dq, dk, dv) to write into, strided or not, apart from the inputs; rows of no segment
    are left as they were there, and zero in gradients allocated here. Offsets that cannot be used: as in
    view_attn_fwd."""
    Lq, Lk, nseg, strides, device = _check_view(cfg, q, k, v, q_offs, k_offs, dev_status)
    H, Hkv = cfg.H, cfg.kv_heads
    _dense(out, "out", (Lq, H, 64), torch.bfloat16, device)
    _dense(lse, "lse", (H, Lq), torch.float32, device)
    _dense(dout, "dout", (Lq, H, 64), torch.bfloat16, device)
    all_rows = grads is None
    if all_rows:
        dq, dk, dv = torch.empty_like(out), _new(k, (Lk, Hkv, 64)), _new(v, (Lk, Hkv, 64))
        strides = (*strides, 0, 0, 0, 0, 0, 0)
    else:
        dq, dk, dv = grads
        strides = (*strides, *_rows(dq, "dq", (Lq, H, 64), _BF16, device),
                   *_rows(dk, "dk", (Lk, Hkv, 64), _BF16, device),
                   *_rows(dv, "dv", (Lk, Hkv, 64), _BF16, device))
    p = cfg._params(Lq, Lk, nseg, all_rows, dev_status, strides)
    workspace = _workspace(workspace, _lib.load().s3r_view_attn_bwd_workspace_bytes(ctypes.byref(p)), q,
                           device)
    _lib.call("s3r_view_attn_bwd", ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
              q_offs.data_ptr(), k_offs.data_ptr(), out.data_ptr(), lse.data_ptr(),
              dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(workspace),
              0 if workspace is None else workspace.numel(), _raw_stream(device))
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
    @once_differentiable
    def backward(ctx, dout):
        dout = _as_rows(dout.to(torch.bfloat16), dout)
        return (*view_attn_bwd(ctx.cfg, *ctx.saved_tensors, dout), None, None, None)
