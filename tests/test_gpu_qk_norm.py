"""GPU tests of the per-head norm with rotation (s3r_qk_norm_rope_fwd / _bwd) against fp64.

Bounds: fp32 arithmetic on values of order 1 (the inputs are standard normal, so xhat is below 8):
a row sum of 64 terms, a reciprocal square root (2 ulp), a cosine and sine (2 ulp of 1, angles
rounded to fp32 after their reduction to half a turn: 2^-23), a handful of products: 40 steps of
2^-24 of the magnitudes |y_a| + |y_b| that enter an output cover them. Then one rounding to the
output's type, 2^-8 (bf16) or 2^-24 (fp32) of the value."""
import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r

import view_ref as R

pytestmark = pytest.mark.gpu
ROUND = {torch.bfloat16: R.BF, torch.float32: R.F32}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def make(L, H, Hk, dtype, norm, rope, seed, dev, pos_top=1000):
    g = torch.Generator().manual_seed(seed)
    x = dict(q=torch.randn((L, H, 64), generator=g).to(dtype).to(dev),
             k=torch.randn((L, Hk, 64), generator=g).to(dtype).to(dev))
    w = {}
    for n in "qk":
        w[n + "_weight"] = None if norm == "none" else (1 + 0.3 * torch.randn(64, generator=g)).to(dev)
        w[n + "_bias"] = (0.3 * torch.randn(64, generator=g)).to(dev) if norm == "layer" else None
    shape = {"none": None, "1d": (L,), "2d": (L, 2)}[rope]
    pos = None if shape is None else torch.randint(-pos_top, pos_top, shape, generator=g,
                                                   dtype=torch.int32).to(dev)
    return x, w, pos


def swapped(y, rope):
    """|y| of a channel and of its partner, added: what enters an output of the rotation."""
    y = y.abs()
    if rope == "none":
        return y
    c = torch.arange(64, device=y.device)
    return y + y[..., c ^ (32 if rope == "1d" else 16)]


SHAPES = [(1, 16, 16), (1, 1, 1), (3, 2, 1), (37, 5, 0), (37, 0, 3), (500, 6, 3), (5000, 1, 1),
          (40000, 2, 2)]


@pytest.mark.parametrize("rope", ["1d", "2d", "none"])
@pytest.mark.parametrize("norm", ["layer", "rms", "none"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L,H,Hk", SHAPES)
def test_forward_and_backward(dev, L, H, Hk, dtype, norm, rope):
    x, w, pos = make(L, H, Hk, dtype, norm, rope, 3, dev)
    cfg = s3r.QKNormConfig(norm=norm, rope=rope, base=100.0 if rope == "2d" else 10000.0)
    out = s3r.qk_norm_rope(cfg, x["q"], x["k"], pos, **w)
    g = torch.Generator().manual_seed(4)
    gtype = torch.float32 if (L + H) % 2 else torch.bfloat16
    up = [torch.randn(t.shape, generator=g).to(gtype).to(dev) for t in out]
    grads = s3r.qk_norm_rope_bwd(cfg, x["q"], x["k"], pos, *up, **w)
    for i, n in enumerate("qk"):
        a = (norm, rope, cfg.base, cfg.eps)
        want = R.qk_norm_rope(x[n], pos, w[n + "_weight"], w[n + "_bias"], *a)
        got = out[i].double()
        err = 40 * R.F32 * swapped(R.turn(want, pos, rope, cfg.base, back=True), rope)
        err = err + ROUND[dtype] * want.abs() + 2.0 ** -21
        assert out[i].dtype == dtype
        assert ((got - want).abs() <= err).all(), f"{n}: {((got - want).abs() - err).max():.3e}"

        dx, dw, db = R.qk_norm_rope_bwd(x[n], pos, w[n + "_weight"], up[i], *a)
        # magnitudes: |h| and the two row means times |xhat|, times r
        xhat, r = R.normed(x[n], norm, cfg.eps)
        dy = R.turn(up[i].double(), pos, rope, cfg.base, back=True)
        h = swapped(dy, rope) * (1.0 if w[n + "_weight"] is None else w[n + "_weight"].double().abs())
        mag = (h + (h * xhat.abs()).mean(-1, keepdim=True) * xhat.abs() + h.mean(-1, keepdim=True)) * r
        got = (grads.q, grads.k)[i].double()
        err = 60 * R.F32 * mag + ROUND[dtype] * dx.abs()
        assert ((got - dx).abs() <= err).all(), f"d{n}: {((got - dx).abs() - err).max():.3e}"
        # a weight's gradient: fp32 sums of at most L H terms, each off by 60 steps
        for name, want_w, terms in (("weight", dw, swapped(dy, rope) * (xhat.abs() + 1)),
                                    ("bias", db, swapped(dy, rope))):
            got_w = getattr(grads, f"{n}_{name}")
            if norm == "none" or (name == "bias" and norm != "layer"):
                assert got_w is None
                continue
            # a lane adds at most 40 + L H / 1000 terms before the fp64 sum of the blocks
            steps = 60 + 40 + x[n].shape[0] * x[n].shape[1] / 100
            err = steps * R.F32 * terms.sum((0, 1)) + R.F32 * want_w.abs()
            assert got_w.dtype == torch.float32
            assert ((got_w.double() - want_w).abs() <= err + 1e-30).all(), f"{n}_{name}"


@pytest.mark.parametrize("top", [2 ** 20, 2 ** 31 - 1])
def test_far_positions_keep_their_angles(dev, top):
    """Angles of positions up to the largest int32: exact to fp32 after the reduction."""
    x, w, _ = make(64, 2, 2, torch.float32, "rms", "1d", 5, dev)
    pos = (top - torch.arange(64, dtype=torch.int32)).to(dev)
    cfg = s3r.QKNormConfig(norm="rms", rope="1d", base=10000.0)
    q, _ = s3r.qk_norm_rope(cfg, x["q"], x["k"], pos, **w)
    want = R.qk_norm_rope(x["q"], pos, w["q_weight"], None, "rms", "1d", 10000.0, cfg.eps)
    # the fp64 angle of 2^31 turns holds 2^31 * 2^-52 of itself on either side: under 2^-20
    assert (q.double() - want).abs().max() <= 1e-5
