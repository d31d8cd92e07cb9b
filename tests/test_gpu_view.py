"""GPU tests of dense attention inside segments (s3r_view_attn_fwd / _bwd) against fp64, within
elementwise bounds that follow from the roundings (view_ref.py)."""
import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r
from sparse_global_attention_s3r_b200 import _lib

import view_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def offs(lens):
    o = [0]
    for x in lens:
        o.append(o[-1] + x)
    return o


def make(lq, lk, H, Hkv, seed, dev, tail=0, gain=1.5):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s, m=1.0: (torch.randn(s, generator=g) * m).to(torch.bfloat16).to(dev)  # noqa: E731
    Lq, Lk = sum(lq) + tail, sum(lk) + tail
    return dict(q=bf(Lq, H, 64, m=gain), k=bf(Lk, Hkv, 64), v=bf(Lk, Hkv, 64),
                dout=bf(Lq, H, 64, m=0.1), qo=offs(lq), ko=offs(lk))


def dev_offs(x, dev):
    return (torch.tensor(x["qo"], dtype=torch.int32, device=dev),
            torch.tensor(x["ko"], dtype=torch.int32, device=dev))


def within(name, got, want, err):
    got = got.double()
    same = got == want  # -inf too
    d = torch.where(same, torch.zeros_like(want), (got - want).abs())
    assert torch.isfinite(d).all(), f"{name}: non-finite"
    over = d - (err + 1e-30)
    assert over.max() <= 0, f"{name}: off by {d.flatten()[over.argmax()]:.3e}, bound {err.flatten()[over.argmax()]:.3e}"


CASES = {  # name: (query lengths, key lengths, H, Hkv, rows past the last segment)
    "one_of_each": ([1], [1], 1, 1, 0),
    "one_query": ([1], [300], 2, 2, 0),
    "one_key": ([300], [1], 2, 2, 0),
    "a_full_tile": ([128], [128], 2, 2, 0),
    "tile_and_one": ([129], [129], 2, 2, 0),
    "block_and_one": ([257], [383], 1, 1, 0),
    "many_key_tiles": ([40], [2000], 2, 1, 0),
    "views": ([300] * 5, [300] * 5, 3, 3, 0),
    "ragged": ([5, 0, 130, 257, 64, 1, 77], [9, 40, 0, 129, 511, 1, 250], 4, 2, 11),
    "shared_by_all": ([200, 70], [150, 260], 6, 1, 3),
    "no_keys_at_all": ([10, 20], [0, 0], 2, 2, 5),
    "no_queries_at_all": ([0, 0], [10, 20], 2, 2, 5),
    "view_1374": ([1374], [1374], 2, 2, 0),
    "long_keys_split": ([3], [9000], 1, 1, 0),
    "long_queries": ([2500], [20], 2, 1, 0),
}


def run_fwd(x, H, Hkv, dev, **kw):
    cfg = s3r.ViewConfig(H=H, Hkv=Hkv, max_q=max(b - a for a, b in zip(x["qo"], x["qo"][1:])),
                         max_k=max(b - a for a, b in zip(x["ko"], x["ko"][1:])), **kw)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), dev_status=word)
    assert s3r.read_device_status(word) == 0
    return cfg, out, lse


@pytest.mark.parametrize("name", list(CASES))
def test_forward(dev, name):
    lq, lk, H, Hkv, tail = CASES[name]
    x = make(lq, lk, H, Hkv, 7, dev, tail)
    _, out, lse = run_fwd(x, H, Hkv, dev)
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"])
    within("lse", lse, ref.lse, ref.lse_err)
    within("out", out, ref.out, ref.out_err)


@pytest.mark.parametrize("name", list(CASES))
def test_backward(dev, name):
    lq, lk, H, Hkv, tail = CASES[name]
    x = make(lq, lk, H, Hkv, 8, dev, tail)
    cfg, out, lse = run_fwd(x, H, Hkv, dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    dq, dk, dv = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse,
                                   x["dout"], dev_status=word)
    assert s3r.read_device_status(word) == 0
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"], dout=x["dout"])
    within("dv", dv, ref.dv, ref.dv_err)
    within("dq", dq, ref.dq, ref.dq_err)
    within("dk", dk, ref.dk, ref.dk_err)


@pytest.mark.parametrize("shape", [([300], [700]), ([5], [700]), ([130, 3], [200, 900])])
@pytest.mark.parametrize("step", [20.0, 100.0, 1000.0, -1000.0])
def test_forward_where_logits_climb_tile_by_tile(dev, shape, step):
    """Key tile t's logits are about step * t above the first's, up to 5,000 above: beyond what a row's
    first reference can hold, so that it has to move, or far below it."""
    x = make(*shape, 2, 2, 21, dev)
    for s in range(len(shape[1])):
        t = torch.arange(shape[1][s], device=dev) // 100
        x["k"][x["ko"][s]:x["ko"][s + 1], :, 0] = (step * t)[:, None].to(torch.bfloat16)
    x["q"][..., 0] = 8.0  # scale 1/8: the channel adds step * t
    _, out, lse = run_fwd(x, 2, 2, dev)
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"])
    within("lse", lse, ref.lse, ref.lse_err)
    within("out", out, ref.out, ref.out_err)


def test_forward_where_only_some_rows_climb(dev):
    """Rows of one warp with and without a far tile, in the middle of the keys and at their cut end."""
    x = make([256], [650], 1, 1, 22, dev)
    x["k"][300, 0] = 0
    x["k"][300, 0, 1] = 64.0
    x["k"][649, 0] = 0
    x["k"][649, 0, 2] = 64.0
    x["q"][3::7, 0, 1] = 40.0   # logit 320 at key 300
    x["q"][5::11, 0, 2] = 60.0  # logit 480 at key 649
    _, out, lse = run_fwd(x, 1, 1, dev)
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"])
    within("lse", lse, ref.lse, ref.lse_err)
    within("out", out, ref.out, ref.out_err)


@pytest.mark.parametrize("key", [0, 1, 2, 3, 4, 17, 40, 127, 128, 200, 299])
def test_nan_and_inf_of_a_key_reach_its_own_segment_only(dev, key):
    """A NaN key makes every row of its segment NaN, whichever way its exponential is computed; rows
    of the other segments, whose tiles may hold the key beyond their end, do not see it."""
    x = make([100, 100, 90], [300, 300, 20], 2, 2, 23, dev)
    x["k"][300 + key, :, 3] = float("nan")
    _, out, lse = run_fwd(x, 2, 2, dev)
    assert out[100:200].isnan().all() and lse[:, 100:200].isnan().all()
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"])
    for rows in (slice(0, 100), slice(200, 290)):
        within("out", out[rows], ref.out[rows], ref.out_err[rows])
        within("lse", lse[:, rows], ref.lse[:, rows], ref.lse_err[:, rows])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_around_a_segment_do_not_reach_it(dev, bad):
    """Everything outside a segment is NaN or infinite: the rows before and after it in every tensor,
    forward and backward."""
    x = make([70, 133, 50], [90, 201, 60], 2, 1, 24, dev, tail=9)
    qs, ks = slice(70, 203), slice(90, 291)
    y = {n: t.clone() for n, t in x.items() if isinstance(t, torch.Tensor)}
    for n in ("q", "dout", "k", "v"):
        keep = qs if n in ("q", "dout") else ks
        y[n][:] = bad
        y[n][keep] = x[n][keep]
    x.update(y)
    cfg, out, lse = run_fwd(x, 2, 1, dev)
    dq, dk, dv = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
    ref = R.attention(x["q"][qs], x["k"][ks], x["v"][ks], [0, 133], [0, 201], dout=x["dout"][qs])
    within("out", out[qs], ref.out, ref.out_err)
    within("dq", dq[qs], ref.dq, ref.dq_err)
    within("dk", dk[ks], ref.dk, ref.dk_err)
    within("dv", dv[ks], ref.dv, ref.dv_err)
