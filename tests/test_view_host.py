"""The dense operators on the host: the exports and argument checks of include/s3r_view.h (every call fails
validation before it touches a device), the torch front end's refusals, and the fp64 references the
GPU tests compare with, against differences of their own forwards and against torch."""
import ctypes
import os
import re

import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r
from sparse_global_attention_s3r_b200 import _lib, view

import view_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, BAD, UNS, WS = (_lib.S3R_OK, _lib.S3R_ERR_INVALID_ARG, _lib.S3R_ERR_UNSUPPORTED,
                    _lib.S3R_ERR_WORKSPACE)
# never dereferenced: validation comes first
A16, A8, A4, A2 = 1 << 20, (1 << 20) + 8, (1 << 20) + 4, (1 << 20) + 2
A256, A16_NOT256 = 1 << 24, (1 << 24) + 16


def test_library_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "s3r_view.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(s3r_[a-z0-9_]+)\s*\(", text))
    assert names == set(_lib.VIEW_EXPORTS)
    for n in names:
        assert hasattr(_lib.load(), n)


def norm_params(**kw):
    p = _lib.QKNormParams(L=10, H=4, Hk=2, d=64, norm=1, rope=2, dtype=0, grad_dtype=0, eps=1e-6, base=100.0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def view_params(**kw):
    p = _lib.ViewParams(Lq=1000, Lk=1000, H=4, Hkv=2, d=64, nseg=3, max_q=400, max_k=400)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def norm_fwd(p, args=None):
    args = args or [A16] * 9
    return _lib.load().s3r_qk_norm_rope_fwd(ctypes.byref(p) if p else None, *args, None)


def norm_bwd(p, args=None, ws=A256, n=1 << 40):
    args = args or [A16] * 10
    return _lib.load().s3r_qk_norm_rope_bwd(ctypes.byref(p) if p else None, *args, ws, n, None)


def view_fwd(p, args=None, ws=A256, n=1 << 40):
    args = args or [A16] * 7
    return _lib.load().s3r_view_attn_fwd(ctypes.byref(p) if p else None, *args, ws, n, None)


def view_bwd(p, args=None, ws=A256, n=1 << 40):
    args = args or [A16] * 11
    return _lib.load().s3r_view_attn_bwd(ctypes.byref(p) if p else None, *args, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=128), UNS), (dict(dtype=7), UNS), (dict(L=-1), BAD), (dict(L=1 << 31), BAD),
    (dict(H=-1), BAD), (dict(H=0, Hk=0), BAD), (dict(norm=3), BAD), (dict(rope=-1), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(base=0.0), BAD), (dict(base=float("nan")), BAD), (dict(base=float("inf")), BAD),
    # strides: below a row, no multiple of 8, rows that overlap, beyond a tensor map's reach
    (dict(q_stride_tok=32, q_stride_head=64), BAD), (dict(q_stride_tok=260, q_stride_head=64), BAD),
    (dict(k_stride_tok=64, k_stride_head=64), BAD), (dict(qo_stride_tok=192, qo_stride_head=64), BAD),
    (dict(ko_stride_tok=1 << 40, ko_stride_head=64), BAD),
    (dict(q_stride_tok=-256, q_stride_head=64), BAD),
])
def test_norm_rejects_bad_parameters(kw, want):
    p = norm_params(**kw)
    assert norm_fwd(p) == want and norm_bwd(p) == want
    assert _lib.load().s3r_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(p)) == 0


def test_norm_rejects_bad_pointers_and_workspaces():
    assert norm_fwd(None) == BAD and norm_bwd(None) == BAD
    for i in range(9):  # q k pos qw qb kw kb q_out k_out
        for bad in (A8 if i != 2 else A2,) + ((None,) if i in (0, 1, 2, 7, 8) else ()):
            a = [A16] * 9
            a[i] = bad
            assert norm_fwd(norm_params(), a) == BAD, i
    for i in range(10):  # q k pos qw kw gq gk dq dk dw
        for bad in (A8 if i != 2 else A2,) + ((None,) if i not in (3, 4) else ()):
            a = [A16] * 10
            a[i] = bad
            assert norm_bwd(norm_params(), a) == BAD, i
    # weights that the norm does not have
    assert norm_fwd(norm_params(norm=2)) == BAD and norm_fwd(norm_params(norm=0)) == BAD
    assert norm_bwd(norm_params(norm=0)) == BAD
    assert norm_bwd(norm_params(grad_dtype=9)) == UNS
    for kw in (dict(dq_stride_tok=64, dq_stride_head=64), dict(dk_stride_tok=100, dk_stride_head=64)):
        assert norm_bwd(norm_params(**kw)) == BAD
    need = _lib.load().s3r_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(norm_params()))
    for ws, n in ((None, need), (A256, need - 1), (A16_NOT256, need)):
        assert norm_bwd(norm_params(), ws=ws, n=n) == WS


@pytest.mark.parametrize("kw,want", [
    (dict(d=32), UNS), (dict(Lq=-1), BAD), (dict(Lk=1 << 31), BAD), (dict(H=0), BAD), (dict(Hkv=0), BAD),
    (dict(Hkv=3), BAD), (dict(H=70000, Hkv=1), BAD), (dict(nseg=0), BAD), (dict(max_q=-1), BAD),
    (dict(max_k=-1), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(q_stride_tok=128, q_stride_head=64), BAD), (dict(k_stride_tok=130, k_stride_head=64), BAD),
    (dict(v_stride_tok=64, v_stride_head=0), BAD), (dict(dq_stride_tok=64, dq_stride_head=64), BAD),
    (dict(dk_stride_tok=64, dk_stride_head=64), BAD), (dict(dv_stride_tok=8, dv_stride_head=8), BAD),
    (dict(dev_status=A2), BAD),
])
def test_attention_rejects_bad_parameters(kw, want):
    p = view_params(**kw)
    assert view_fwd(p) == want and view_bwd(p) == want
    assert _lib.load().s3r_view_attn_bwd_workspace_bytes(ctypes.byref(p)) == 0


def test_attention_rejects_bad_pointers_and_workspaces():
    assert view_fwd(None) == BAD and view_bwd(None) == BAD
    for i in range(7):  # q k v q_offs k_offs out lse (lse may be null)
        for bad in (A8 if i not in (3, 4) else A2,) + ((None,) if i != 6 else ()):
            a = [A16] * 7
            a[i] = bad
            assert view_fwd(view_params(), a) == BAD, i
    for i in range(11):  # q k v q_offs k_offs out lse dout dq dk dv
        for bad in (A8 if i not in (3, 4) else A2, None):
            a = [A16] * 11
            a[i] = bad
            assert view_bwd(view_params(), a) == BAD, i
    need = _lib.load().s3r_view_attn_bwd_workspace_bytes(ctypes.byref(view_params()))
    for ws, n in ((None, need), (A256, need - 1), (A16_NOT256, need)):
        assert view_bwd(view_params(), ws=ws, n=n) == WS
    # few rows over long keys: the forward's pieces need a workspace too
    p = view_params(Lq=1, Lk=100000, nseg=1, max_q=1, max_k=100000)
    need = _lib.load().s3r_view_attn_workspace_bytes(ctypes.byref(p))
    assert need > 0
    for ws, n in ((None, need), (A256, need - 1), (A16_NOT256, need)):
        assert view_fwd(p, ws=ws, n=n) == WS
    p = view_params(Lq=100000, Lk=100000, nseg=100, max_q=1000, max_k=1000)
    assert _lib.load().s3r_view_attn_workspace_bytes(ctypes.byref(p)) == 0


def test_front_end_refuses_before_any_call():
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    o = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        s3r.view_attn_fwd(s3r.ViewConfig(H=2), q, q, q, o, o)
    with pytest.raises(ValueError, match="heads"):
        s3r.view_attn_fwd(s3r.ViewConfig(H=3), q, q, q, o, o)
    with pytest.raises(ValueError, match=r"\[L, H, 64\]"):
        s3r.view_attn_fwd(s3r.ViewConfig(H=2), q[..., :32], q, q, o, o)
    with pytest.raises(ValueError, match="CUDA"):
        s3r.qk_norm_rope(s3r.QKNormConfig(rope="none"), q, q)
    with pytest.raises(ValueError, match="norm 'batch'"):
        s3r.qk_norm_rope(s3r.QKNormConfig(norm="batch"), q, q)
    with pytest.raises(ValueError, match="same tokens"):
        s3r.qk_norm_rope(s3r.QKNormConfig(rope="none"), q, q[:3])
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        s3r.qk_norm_rope(s3r.QKNormConfig(rope="none"), q.half(), q.half())
    with pytest.raises(ValueError, match="positive"):
        s3r.view_positions(0, 3, 3)


def test_view_positions():
    pos = s3r.view_positions(2, 2, 3, special=2)
    one = [[0, 0], [0, 0], [1, 1], [1, 2], [1, 3], [2, 1], [2, 2], [2, 3]]
    assert pos.dtype == torch.int32 and pos.tolist() == one * 2


def test_attention_reference_against_torch_and_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    qo, ko, H, Hkv = [0, 3, 3, 7], [0, 4, 6, 9], 4, 2
    q, k, v, do = r(8, H, 64), r(9, Hkv, 64), r(9, Hkv, 64), r(8, H, 64)
    ref = R.attention(q, k, v, qo, ko, 0.2, do)
    a, b, c = (t.clone().requires_grad_() for t in (q, k, v))
    for s in (0, 2):
        x = [t.transpose(0, 1) for t in (a[qo[s]:qo[s + 1]], b[ko[s]:ko[s + 1]].repeat_interleave(2, 1),
                                         c[ko[s]:ko[s + 1]].repeat_interleave(2, 1))]
        out = torch.nn.functional.scaled_dot_product_attention(*x, scale=0.2).transpose(0, 1)
        torch.testing.assert_close(ref.out[qo[s]:qo[s + 1]], out.detach())
        out.backward(do[qo[s]:qo[s + 1]])
    for got, leaf in ((ref.dq, a), (ref.dk, b), (ref.dv, c)):
        torch.testing.assert_close(got, leaf.grad)
    assert (ref.out[7:] == 0).all() and (ref.lse[:, 7:] == -torch.inf).all()
    # central differences along a direction, error h^2 of a third derivative of order 1
    h, d = 1e-5, [r(*t.shape) for t in (q, k, v)]
    f = lambda e: (R.attention(q + e * d[0], k + e * d[1], v + e * d[2], qo, ko, 0.2).out * do).sum()  # noqa: E731
    want = sum((x * y).sum() for x, y in zip((ref.dq, ref.dk, ref.dv), d))
    assert abs((f(h) - f(-h)) / (2 * h) - want) <= 1e-6 * abs(want) + 1e-6


@pytest.mark.parametrize("norm", ["layer", "rms", "none"])
@pytest.mark.parametrize("rope", ["1d", "2d", "none"])
def test_norm_reference_against_torch_and_differences(norm, rope):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, up = r(5, 3, 64), r(64), r(64), r(5, 3, 64)
    pos = torch.randint(-50, 50, (5, 2) if rope == "2d" else (5,), generator=g, dtype=torch.int32)
    w_, b_ = (None if norm == "none" else w), (b if norm == "layer" else None)
    if norm == "layer" and rope == "none":
        torch.testing.assert_close(R.qk_norm_rope(x, pos, w, b, norm, rope, 100.0, 1e-6),
                                   torch.nn.functional.layer_norm(x, (64,), w, b, 1e-6))
    # a rotation keeps every pair's length; position 0 turns nothing
    y = R.turn(x, pos, rope, 100.0)
    torch.testing.assert_close(y.square().sum(-1), x.square().sum(-1))
    torch.testing.assert_close(R.turn(y, pos, rope, 100.0, back=True), x)
    torch.testing.assert_close(R.turn(x, torch.zeros_like(pos), rope, 100.0), x)
    dx, dw, db = R.qk_norm_rope_bwd(x, pos, w_, up, norm, rope, 100.0, 1e-6)
    f = lambda x, w, b: (R.qk_norm_rope(x, pos, w, b, norm, rope, 100.0, 1e-6) * up).sum()  # noqa: E731
    h, d = 1e-5, r(*x.shape)
    assert abs((f(x + h * d, w_, b_) - f(x - h * d, w_, b_)) / (2 * h) - (dx * d).sum()) <= 1e-5
    if w_ is not None:
        e = r(64)
        assert abs((f(x, w + h * e, b_) - f(x, w - h * e, b_)) / (2 * h) - (dw * e).sum()) <= 1e-5
    if b_ is not None:
        e = r(64)
        assert abs((f(x, w, b + h * e) - f(x, w, b - h * e)) / (2 * h) - (db * e).sum()) <= 1e-5


def test_workspaces_go_by_the_segments_not_by_the_tensors():
    """Partial results of split walks are for nseg segments of the greatest length; only D (4 bytes a
    query row and head) goes by the tensor."""
    lib = _lib.load()

    def sizes(L, **kw):
        p = ctypes.byref(view_params(Lq=L, Lk=L, H=2, Hkv=2, nseg=2, max_q=30, max_k=2300, **kw))
        return lib.s3r_view_attn_workspace_bytes(p), lib.s3r_view_attn_bwd_workspace_bytes(p)

    small, large = sizes(4600), sizes(4_600_000)
    assert small[0] == large[0] > 0
    assert 0 < large[1] - small[1] <= 4 * 2 * 4_600_000
    assert small[0] < 1 << 22 and small[1] - 4 * 2 * 4600 < 64 << 20


@pytest.mark.parametrize("kw", [
    dict(nseg=2 ** 31 - 1), dict(nseg=1 << 24, H=256, Hkv=1),
    dict(Lq=2 ** 31 - 1, max_q=2 ** 31 - 1, H=4096, Hkv=1, nseg=1),
    dict(Lq=2 ** 31 - 1, Lk=2 ** 31 - 1, max_q=2 ** 31 - 1, max_k=2 ** 31 - 1, H=65535, Hkv=1, nseg=2 ** 31 - 1),
])
def test_attention_refuses_more_blocks_than_a_grid_holds(kw):
    p = view_params(**kw)
    assert view_fwd(p) == BAD and view_bwd(p) == BAD
    assert _lib.load().s3r_view_attn_workspace_bytes(ctypes.byref(p)) == 0


def test_front_end_refuses_a_workspace_that_is_not_the_devices():
    with pytest.raises(ValueError, match="workspace is on cpu"):
        view._workspace(torch.zeros(1024, dtype=torch.uint8), 256, torch.zeros(1), 0)


@pytest.mark.parametrize("scale", [0.0, -0.125, float("nan"), float("inf")])
def test_front_end_refuses_a_scale_that_is_not_positive(scale):
    with pytest.raises(ValueError, match="scale must be positive"):
        s3r.ViewConfig(H=2, scale=scale)._params(4, 4, 1, True, None, (0,) * 12)
