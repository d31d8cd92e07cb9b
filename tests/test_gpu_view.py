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
