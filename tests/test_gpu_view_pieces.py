"""GPU tests of dense attention whose walk over the keys is split into pieces (few queries over many keys),
against fp64, within the bounds of view_ref.py."""
import ctypes

import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r
from sparse_global_attention_s3r_b200 import _lib

import view_ref as R
from test_gpu_view import dev_offs, make, run_fwd, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def is_split(x, H, Hkv):
    """Whether the forward's walk and the one of dq's kernel are split: partial results need room."""
    longest = [max(b - a for a, b in zip(o, o[1:])) for o in (x["qo"], x["ko"])]
    cfg = s3r.ViewConfig(H=H, Hkv=Hkv, max_q=longest[0], max_k=longest[1])
    Lq, Lk = x["q"].shape[0], x["k"].shape[0]
    p = ctypes.byref(cfg._params(Lq, Lk, len(x["qo"]) - 1, True, None, (0,) * 12))
    d = -(-Lq * H * 4 // 256) * 256
    return (_lib.load().s3r_view_attn_workspace_bytes(p) > 0
            and _lib.load().s3r_view_attn_bwd_workspace_bytes(p) > max(d, 256))


@pytest.mark.parametrize("keys", [2000, 9000])
@pytest.mark.parametrize("queries", [1, 40, 200])
def test_far_logits_in_every_key_tile(dev, queries, keys):
    """One key tile at a time holds a key whose logit with every third row is 64, about 85 octaves above
    what a row sees first: the row's reference has to move in that tile, be it the last one of any piece."""
    x = make([queries], [keys], 1, 1, 71, dev)
    assert is_split(x, 1, 1)
    x["q"][::3, 0, 0] = 8.0
    plain = x["k"].clone()
    for t in range(-(-keys // 128)):
        x["k"].copy_(plain)
        at = min(t * 128 + 100, keys - 1)
        x["k"][at, 0] = 0
        x["k"][at, 0, 0] = 64.0
        _, out, lse = run_fwd(x, 1, 1, dev)
        ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"])
        within(f"lse, tile {t}", lse, ref.lse, ref.lse_err)
        within(f"out, tile {t}", out, ref.out, ref.out_err)


@pytest.mark.parametrize("step", [20.0, 100.0, 1000.0])
def test_logits_climb_from_piece_to_piece(dev, step):
    """Forward and backward where every hundred keys lift the logits by `step`."""
    x = make([40], [5000], 1, 1, 72, dev)
    assert is_split(x, 1, 1)
    t = torch.arange(5000, device=dev) // 100
    x["k"][:, 0, 0] = (step * t).to(torch.bfloat16)
    x["q"][..., 0] = 8.0
    cfg, out, lse = run_fwd(x, 1, 1, dev)
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"], dout=x["dout"])
    within("lse", lse, ref.lse, ref.lse_err)
    within("out", out, ref.out, ref.out_err)
    grads = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
    for g, n in zip(grads, ("dq", "dk", "dv")):
        within(n, g, getattr(ref, n), getattr(ref, n + "_err"))


@pytest.mark.parametrize("gain", [1.5, 6.0])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1)])
def test_short_segments_beside_a_split_one(dev, H, Hkv, gain):
    """Segments of one tile and of two beside one whose walk is split, with ordinary and with concentrated
    softmax rows: D of up to 256 keys is the sum of P dP there too (view_ref.py's bound)."""
    x = make([3, 40, 20, 7], [5000, 100, 200, 1], H, Hkv, 73, dev, tail=5, gain=gain)
    assert is_split(x, H, Hkv)
    cfg, out, lse = run_fwd(x, H, Hkv, dev)
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"], dout=x["dout"])
    within("lse", lse, ref.lse, ref.lse_err)
    within("out", out, ref.out, ref.out_err)
    grads = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
    for g, n in zip(grads, ("dq", "dk", "dv")):
        within(n, g, getattr(ref, n), getattr(ref, n + "_err"))


def test_gradients_of_short_segments_do_not_go_by_the_bounds(dev):
    """The same segments with bounds that are tight and with bounds that have the walks split: dq is the
    same bit by bit, since one piece walks the whole of a short segment."""
    x = make([30, 50], [250, 130], 1, 1, 74, dev)
    cfg, out, lse = run_fwd(x, 1, 1, dev)
    far = {n: torch.cat([x[n], x[n].new_zeros((5000, 1, 64))]) for n in "kv"}
    wide = s3r.ViewConfig(H=1, max_q=50, max_k=5000)
    args = *dev_offs(x, dev), out, lse, x["dout"]
    tight = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *args)
    loose = s3r.view_attn_bwd(wide, x["q"], far["k"], far["v"], *args)
    assert torch.equal(tight[0], loose[0])


@pytest.mark.parametrize("queries,keys,split", [(200, 300, False), (300, 130, False), (40, 5000, True),
                                                (200, 5000, True)])
@pytest.mark.parametrize("part", [0.0, 0.4, 0.999])
def test_nan_of_a_key_in_both_tiles_and_in_any_piece(dev, queries, keys, split, part):
    """More than 128 query rows, and a walk in pieces: a NaN key makes all rows of its segment NaN, and
    the other segment's none."""
    x = make([queries, 30], [keys, 100], 1, 1, 75, dev)
    assert is_split(x, 1, 1) == split
    x["k"][int(part * keys), 0, 5] = float("nan")
    _, out, lse = run_fwd(x, 1, 1, dev)
    assert out[:queries].isnan().all() and lse[:, :queries].isnan().all()
    ref = R.attention(x["q"][queries:], x["k"][keys:], x["v"][keys:], [0, 30], [0, 100])
    within("out", out[queries:], ref.out, ref.out_err)
    within("lse", lse[:, queries:], ref.lse, ref.lse_err)


def test_unusable_segments_beside_split_ones_are_nan_in_allocated_results(dev):
    """A bound that the middle of three segments exceeds, in walks that are split and joined: its rows are
    NaN, the others' as without it."""
    lk = [2000, 2001, 2000]
    x = make([50, 40, 30], lk, 1, 1, 76, dev)
    assert is_split(x, 1, 1)
    o, word = dev_offs(x, dev), torch.zeros(1, dtype=torch.int32, device=dev)
    good, tight = (s3r.ViewConfig(H=1, max_q=50, max_k=n) for n in (2001, 2000))  # equal tiles and pieces
    want = s3r.view_attn_fwd(good, x["q"], x["k"], x["v"], *o)
    got = s3r.view_attn_fwd(tight, x["q"], x["k"], x["v"], *o, dev_status=word)
    assert s3r.read_device_status(word) == _lib.S3R_DEV_BAD_INDEX
    g_want = s3r.view_attn_bwd(good, x["q"], x["k"], x["v"], *o, *want, x["dout"])
    g_got = s3r.view_attn_bwd(tight, x["q"], x["k"], x["v"], *o, *want, x["dout"])
    for a, b, offs in zip((got[0], got[1].t(), *g_got), (want[0], want[1].t(), *g_want),
                          ("qo", "qo", "qo", "ko", "ko")):
        s = slice(x[offs][1], x[offs][2])
        assert torch.isnan(a[s]).all()
        same = torch.ones(a.shape[0], dtype=torch.bool, device=dev)
        same[s] = False
        assert torch.equal(a[same], b[same])
