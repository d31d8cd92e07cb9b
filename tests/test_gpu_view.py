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


def packed(x, dev, spare=0):
    """q, k, v as views of one [L, 3 (+ spare), H, 64] projection."""
    L, H = x["q"].shape[:2]
    buf = torch.full((L, 3 + spare, H, 64), float("nan"), dtype=torch.bfloat16, device=dev)
    for i, n in enumerate("qkv"):
        buf[:, i] = x[n]
    return buf


def test_strided_inputs_and_outputs(dev):
    """Views of a packed projection in, gradients into the same layout; neighbours stay as they were."""
    H = 3
    x = make([200, 131], [200, 131], H, H, 31, dev)
    cfg = s3r.ViewConfig(H=H, max_q=200, max_k=200)
    offs_ = dev_offs(x, dev)
    buf = packed(x, dev, spare=1)
    out, lse = s3r.view_attn_fwd(cfg, buf[:, 0], buf[:, 1], buf[:, 2], *offs_)
    want, want_lse = s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *offs_)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    dbuf = torch.full_like(buf, 7.0)
    s3r.view_attn_bwd(cfg, buf[:, 0], buf[:, 1], buf[:, 2], *offs_, out, lse, x["dout"],
                      grads=(dbuf[:, 0], dbuf[:, 1], dbuf[:, 2]))
    grads = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *offs_, out, lse, x["dout"])
    for i in range(3):
        assert torch.equal(dbuf[:, i], grads[i])
    assert (dbuf[:, 3] == 7).all()
    # head-major storage: heads outermost
    hm = {n: x[n].transpose(0, 1).contiguous().transpose(0, 1) for n in "qkv"}
    out2, _ = s3r.view_attn_fwd(cfg, hm["q"], hm["k"], hm["v"], *offs_)
    assert torch.equal(out2, want)


def test_rows_past_the_last_segment(dev):
    """Left as they were in what the caller passes, zero (lse -inf) in what the call allocates."""
    x = make([40, 90], [60, 70], 2, 1, 32, dev, tail=300)
    cfg, out, lse = run_fwd(x, 2, 1, dev)
    assert (out[130:] == 0).all() and (lse[:, 130:] == -torch.inf).all()
    mine = torch.full_like(out, 3.0), torch.full_like(lse, 5.0)
    s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out=mine[0], lse=mine[1])
    assert torch.equal(mine[0][:130], out[:130]) and (mine[0][130:] == 3).all()
    assert torch.equal(mine[1][:, :130], lse[:, :130]) and (mine[1][:, 130:] == 5).all()
    args = (cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
    g = s3r.view_attn_bwd(*args)
    assert all((t[130:] == 0).all() for t in g)
    mine = tuple(torch.full_like(t, 3.0) for t in g)
    s3r.view_attn_bwd(*args, grads=mine)
    for a, b in zip(g, mine):
        assert torch.equal(a[:130], b[:130]) and (b[130:] == 3).all()


def test_gap_before_the_first_segment_is_left_alone(dev):
    x = make([50], [70], 2, 2, 33, dev)
    y = {n: torch.cat([torch.full_like(x[n][:10], float("inf")), x[n]]) for n in ("q", "k", "v", "dout")}
    o = [torch.tensor(v, dtype=torch.int32, device=dev) for v in ([10, 60], [10, 80])]
    cfg = s3r.ViewConfig(H=2, max_q=50, max_k=70)
    out, lse = torch.full_like(y["q"], 3.0), torch.full((2, 60), 5.0, device=dev)
    s3r.view_attn_fwd(cfg, y["q"], y["k"], y["v"], *o, out=out, lse=lse)
    want, _ = s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev))
    assert torch.equal(out[10:], want) and (out[:10] == 3).all() and (lse[:, :10] == 5).all()


BAD = [  # query and key offsets of two segments, the query rows whose segment cannot be used
    ([0, 50, 40], [0, 30, 60], slice(50, 100)),
    ([0, 50, 101], [0, 30, 60], slice(50, 100)),
    ([0, 50, 90], [0, 30, 61], slice(50, 100)),
    ([-1, 50, 90], [0, 30, 60], slice(0, 50)),
    ([0, 50, 90], [0, -5, 60], slice(0, 100)),
]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("qo,ko,rows", BAD)
def test_unusable_offsets_are_reported_and_their_rows_not_written(dev, qo, ko, rows, split):
    """split: one head and bounds that have the walks split into pieces and joined."""
    H = 1 if split else 2
    x = make([50, 50], [30, 30], H, H, 34, dev)
    if split:  # the same offsets a thousand keys on, so that the walk is long enough to be split
        x["k"], x["v"] = (torch.cat([x[n]] + [x[n][:50]] * 40) for n in "kv")
        ko = [ko[0], ko[1], ko[2] if ko[2] <= 60 else x["k"].shape[0] + 1]
    o = [torch.tensor(v, dtype=torch.int32, device=dev) for v in (qo, ko)]
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = torch.full_like(x["q"], 3.0), torch.full((H, 100), 5.0, device=dev)
    cfg = s3r.ViewConfig(H=H)
    s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *o, out=out, lse=lse, dev_status=word)
    assert s3r.read_device_status(word) == _lib.S3R_DEV_BAD_INDEX
    assert (out[rows] == 3).all() and (lse[:, rows] == 5).all()
    grads = tuple(torch.full_like(x[n], 3.0) for n in "qkv")
    s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *o, out, lse, x["dout"], grads=grads, dev_status=word)
    assert s3r.read_device_status(word) == _lib.S3R_DEV_BAD_INDEX
    assert (grads[0][rows] == 3).all()


def test_a_segment_longer_than_the_config_says_is_reported(dev):
    x = make([50, 50], [30, 30], 2, 2, 34, dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    for cfg in (s3r.ViewConfig(H=2, max_q=49), s3r.ViewConfig(H=2, max_k=29)):
        s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), dev_status=word)
        assert s3r.read_device_status(word) == _lib.S3R_DEV_BAD_INDEX


@pytest.mark.parametrize("name", ["ragged", "long_keys_split", "long_queries"])
def test_equal_calls_give_equal_bits(dev, name):
    lq, lk, H, Hkv, tail = CASES[name]
    x = make(lq, lk, H, Hkv, 35, dev, tail)
    cfg, out, lse = run_fwd(x, H, Hkv, dev)
    args = (cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
    first = s3r.view_attn_bwd(*args)
    for _ in range(5):
        _, o2, l2 = run_fwd(x, H, Hkv, dev)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert all(torch.equal(a, b) for a, b in zip(first, s3r.view_attn_bwd(*args)))


def test_two_streams_at_once(dev):
    xs = [make([500, 300], [500, 300], 4, 4, 36 + i, dev) for i in range(2)]
    want = [run_fwd(x, 4, 4, dev)[1:] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (x, st) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(st):
                cfg = s3r.ViewConfig(H=4, max_q=500, max_k=500)
                out, lse = s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev))
                g = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
                got[i].append((out, *g))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(r[0], want[i][0]) for r in got[i])
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, got[i][0]))


def test_two_captured_graphs_replayed_with_new_contents(dev):
    """Forward and backward in a graph each, with a split walk (workspaces), replayed in turn on other
    inputs and other offsets."""
    graphs = []
    for seed in (41, 42):
        x = make([3, 40], [4000, 900], 1, 1, seed, dev)
        o = dev_offs(x, dev)
        cfg = s3r.ViewConfig(H=1, max_q=64, max_k=4900)
        s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *o)  # first use outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = s3r.view_attn_fwd(cfg, x["q"], x["k"], x["v"], *o)
            grads = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *o, out, lse, x["dout"])
        graphs.append((graph, x, o, out, lse, grads))
    for turn in range(2):
        for graph, x, o, *_ in graphs:
            y = make([3, 40], [4000, 900], 1, 1, 50 + turn, dev)
            for n in ("q", "k", "v", "dout"):
                x[n].copy_(y[n])
            if turn:
                x["qo"], x["ko"] = [0, 20, 43], [0, 1500, 4900]
                for t, v in zip(o, (x["qo"], x["ko"])):
                    t.copy_(torch.tensor(v, dtype=torch.int32))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, x, _, out, lse, grads in graphs:
            ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"], dout=x["dout"])
            within("out", out, ref.out, ref.out_err)
            for g, n in zip(grads, ("dq", "dk", "dv")):
                within(n, g, getattr(ref, n), getattr(ref, n + "_err"))


def test_bounded_wait_timeout_is_reported_and_the_context_survives(dev):
    x = make([300], [300], 2, 2, 43, dev)
    cfg, out, lse = run_fwd(x, 2, 2, dev)
    args = (x["q"], x["k"], x["v"], *dev_offs(x, dev))
    slow = s3r.ViewConfig(H=2, max_q=300, max_k=300, test_timeout=True)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    s3r.view_attn_fwd(slow, *args, dev_status=word)
    assert s3r.read_device_status(word) & _lib.S3R_DEV_TIMEOUT
    s3r.view_attn_bwd(slow, *args, out, lse, x["dout"], dev_status=word)
    assert s3r.read_device_status(word) & _lib.S3R_DEV_TIMEOUT
    _, o2, l2 = run_fwd(x, 2, 2, dev)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_empty_tensors(dev):
    e = lambda n: torch.empty((n, 2, 64), dtype=torch.bfloat16, device=dev)  # noqa: E731
    z = torch.zeros(2, dtype=torch.int32, device=dev)
    cfg = s3r.ViewConfig(H=2)
    out, lse = s3r.view_attn_fwd(cfg, e(0), e(0), e(0), z, z)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    q = torch.randn((5, 2, 64), device=dev).to(torch.bfloat16)
    o5 = torch.tensor([0, 5], dtype=torch.int32, device=dev)
    out, lse = s3r.view_attn_fwd(cfg, q, e(0), e(0), o5, z)
    assert (out == 0).all() and (lse == -torch.inf).all()
    dq, dk, dv = s3r.view_attn_bwd(cfg, q, e(0), e(0), o5, z, out, lse, q)
    assert (dq == 0).all() and dk.shape == (0, 2, 64)
    dq, dk, dv = s3r.view_attn_bwd(cfg, e(0), q, q, z, o5, e(0), lse[:, :0].contiguous(), e(0))
    assert (dk == 0).all() and (dv == 0).all()


def test_rows_beyond_32_bit_element_offsets(dev):
    """A cache of 2.2 million tokens of 16 heads, 2^31 elements before its end."""
    L, H = 2_200_000, 16
    g = torch.Generator(device=dev).manual_seed(44)
    k = torch.randn((L, H, 64), generator=g, device=dev, dtype=torch.bfloat16)
    lo = L - 777
    o = [torch.tensor(v, dtype=torch.int32, device=dev) for v in ([0, 30], [lo, L])]
    q = torch.randn((30, H, 64), generator=g, device=dev, dtype=torch.bfloat16)
    cfg = s3r.ViewConfig(H=H, max_q=30, max_k=777)
    out, lse = s3r.view_attn_fwd(cfg, q, k, k, *o)
    ref = R.attention(q, k[lo:], k[lo:], [0, 30], [0, 777], dout=q)
    within("out", out, ref.out, ref.out_err)
    # the same rows as queries and gradients at the far end
    o = [torch.tensor(v, dtype=torch.int32, device=dev) for v in ([lo, L], [0, 30])]
    cfg = s3r.ViewConfig(H=H, max_q=777, max_k=30)
    out, lse = torch.empty_like(k), torch.empty((H, L), device=dev)
    s3r.view_attn_fwd(cfg, k, q, q, *o, out=out, lse=lse)
    ref = R.attention(k[lo:], q, q, [0, 777], [0, 30], dout=k[lo:])
    within("out", out[lo:], ref.out, ref.out_err)
    dq = torch.empty_like(k)
    dkv = torch.empty_like(q), torch.empty_like(q)
    s3r.view_attn_bwd(cfg, k, q, q, *o, out, lse, k, grads=(dq, *dkv))
    within("dq", dq[lo:], ref.dq, ref.dq_err)
    within("dk", dkv[0], ref.dk, ref.dk_err)
    within("dv", dkv[1], ref.dv, ref.dv_err)


@pytest.mark.parametrize("seed", range(12))
def test_random_layouts(dev, seed):
    """Seeded layouts over every axis: segments, lengths from zero on, heads, tails, scale."""
    import random
    r = random.Random(seed)
    n, Hkv = r.randint(1, 9), r.choice([1, 2, 3])
    H = Hkv * r.choice([1, 2, 3])
    top = r.choice([3, 40, 150, 600])
    lq = [r.choice([0, 1, r.randint(1, top), top]) for _ in range(n)]
    lk = [r.choice([0, 1, r.randint(1, top), top]) for _ in range(n)]
    tail, scale = r.choice([0, 5]), r.choice([None, 0.03, 0.4])
    x = make(lq, lk, H, Hkv, 60 + seed, dev, tail)
    if x["q"].shape[0] == 0 or x["k"].shape[0] == 0:
        pytest.skip("an empty tensor: its own test")
    cfg, out, lse = run_fwd(x, H, Hkv, dev, scale=scale)
    ref = R.attention(x["q"], x["k"], x["v"], x["qo"], x["ko"], scale or 0.125, dout=x["dout"])
    within("out", out, ref.out, ref.out_err)
    within("lse", lse, ref.lse, ref.lse_err)
    grads = s3r.view_attn_bwd(cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev), out, lse, x["dout"])
    for g, name in zip(grads, ("dq", "dk", "dv")):
        within(name, g, getattr(ref, name), getattr(ref, name + "_err"))


def test_few_rows_of_large_tensors(dev):
    """A few rows in use of tensors of 300,000: the workspaces go by the rows in use, and the walks over
    the many keys are split; the rest of an allocated result is zero."""
    L = 300_000
    g = torch.Generator(device=dev).manual_seed(70)
    t = [torch.randn((L, 2, 64), generator=g, device=dev).to(torch.bfloat16) for _ in range(4)]
    o = [torch.tensor(v, dtype=torch.int32, device=dev) for v in ([0, 20, 50], [0, 700, 3000])]
    cfg = s3r.ViewConfig(H=2, max_q=30, max_k=2300)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    out, lse = s3r.view_attn_fwd(cfg, *t[:3], *o)
    grads = s3r.view_attn_bwd(cfg, *t[:3], *o, out, lse, t[3])
    # out, three gradients, lse and D, and the partial sums of 2 * 30 and 2 * 2,300 rows
    assert torch.cuda.max_memory_allocated() - before <= 4 * t[0].nbytes + 2 * lse.nbytes + (64 << 20)
    ref = R.attention(*(x[:3000] for x in t[:3]), [0, 20, 50], [0, 700, 3000], dout=t[3][:3000])
    within("out", out[:50], ref.out[:50], ref.out_err[:50])
    assert (out[50:] == 0).all() and (lse[:, 50:] == -torch.inf).all()
    for x, n, rows in zip(grads, ("dq", "dk", "dv"), (50, 3000, 3000)):
        within(n, x[:rows], getattr(ref, n)[:rows], getattr(ref, n + "_err")[:rows])
        assert (x[rows:] == 0).all()


def test_unfit_workspaces_are_refused(dev):
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=dev)
    k = torch.zeros((5000, 1, 64), dtype=torch.bfloat16, device=dev)
    qo, ko = (torch.tensor([0, n], dtype=torch.int32, device=dev) for n in (1, 5000))
    cfg = s3r.ViewConfig(H=1)
    out, lse = s3r.view_attn_fwd(cfg, q, k, k, qo, ko)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=dev)
    for bad in (ws.cpu(), ws[:256], ws[16:], ws[::2], ws.view(torch.float32)):
        with pytest.raises(ValueError, match="workspace"):
            s3r.view_attn_fwd(cfg, q, k, k, qo, ko, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            s3r.view_attn_bwd(cfg, q, k, k, qo, ko, out, lse, q, workspace=bad)
    assert (s3r.view_attn_fwd(cfg, q, k, k, qo, ko, workspace=ws)[0] == 0).all()


@pytest.mark.parametrize("before,after", [(10, 0), (1, 700), (5000, 9000)])
def test_rows_of_no_segment_in_allocated_results(dev, before, after):
    """Offsets of a few segments out of a longer list: the rows around them are 0, and -inf in lse."""
    x = make([50, 20], [70, 300], 2, 1, 35, dev)
    pad = lambda t: torch.cat([t.new_full((before, *t.shape[1:]), float("nan")), t,  # noqa: E731
                               t.new_full((after, *t.shape[1:]), float("nan"))])
    y = {n: pad(x[n]) for n in ("q", "k", "v", "dout")}
    o = [t + before for t in dev_offs(x, dev)]
    cfg = s3r.ViewConfig(H=2, Hkv=1, max_q=50, max_k=300)
    args = cfg, x["q"], x["k"], x["v"], *dev_offs(x, dev)
    want = s3r.view_attn_fwd(*args)
    grads = s3r.view_attn_bwd(*args, *want, x["dout"])
    got = s3r.view_attn_fwd(cfg, y["q"], y["k"], y["v"], *o)
    back = s3r.view_attn_bwd(cfg, y["q"], y["k"], y["v"], *o, *got, y["dout"])
    for a, b in zip((got[0], got[1].t(), *back), (want[0], want[1].t(), *grads)):
        n = b.shape[0]
        assert torch.equal(a[before:before + n], b)
        rest = torch.cat([a[:before], a[before + n:]])
        assert (rest == (-torch.inf if a.dtype == torch.float32 else 0)).all()


@pytest.mark.parametrize("split", [False, True])
def test_unusable_segments_are_nan_in_allocated_results(dev, split):
    """A bound that the middle segment exceeds: its rows are NaN, whatever reads them without the
    status word; the others' are as without it."""
    lk = [600, 601, 600] if split else [60, 61, 60]
    x = make([50, 40, 30], lk, 1, 1, 36, dev)
    o, word = dev_offs(x, dev), torch.zeros(1, dtype=torch.int32, device=dev)
    good, tight = (s3r.ViewConfig(H=1, max_q=50, max_k=n) for n in (lk[1], lk[0]))  # equal tiles and pieces
    want = s3r.view_attn_fwd(good, x["q"], x["k"], x["v"], *o)
    got = s3r.view_attn_fwd(tight, x["q"], x["k"], x["v"], *o, dev_status=word)
    assert s3r.read_device_status(word) == _lib.S3R_DEV_BAD_INDEX
    g_want = s3r.view_attn_bwd(good, x["q"], x["k"], x["v"], *o, *want, x["dout"])
    g_got = s3r.view_attn_bwd(tight, x["q"], x["k"], x["v"], *o, *want, x["dout"])
    for a, b, offs in zip((got[0], got[1].t(), *g_got), (want[0], want[1].t(), *g_want), ("qo", "qo", "qo", "ko", "ko")):
        s = slice(x[offs][1], x[offs][2])
        assert torch.isnan(a[s]).all()
        same = torch.ones(a.shape[0], dtype=torch.bool, device=dev)
        same[s] = False
        assert torch.equal(a[same], b[same])
