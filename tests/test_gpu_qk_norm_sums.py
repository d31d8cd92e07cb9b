"""GPU tests of what the per-head norm's gradient promises beside its values: every row counted once in the
weights' gradients, equal bits on equal calls, gradients written over the inputs, several streams, and
captured calls."""
import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L,H,Hk", [(1, 1, 1), (37, 5, 3), (500, 6, 3), (5000, 1, 1), (9999, 3, 1),
                                    (40000, 2, 2), (5001, 16, 16)])
def test_every_row_counts_once_in_the_weights_gradients(dev, L, H, Hk, dtype):
    """Rows of +-1 have xhat = +-1 (within 2^-22), and without a rotation a weight's gradient is a sum of
    +-1, +-2 and +-3: an integer, so that a row left out or counted twice is off by 1 at least. The bias's
    is exact: its partial sums are integers below 2^24."""
    g = torch.Generator(device=dev).manual_seed(5)

    def rows(n):
        up = torch.randint(1, 4, (L, n, 64), generator=g, device=dev)
        sign = torch.randint(0, 2, (2, L, n, 64), generator=g, device=dev) * 2 - 1
        # half of each sign: the layer norm's mean is 0
        x = torch.where(torch.rand((L, n, 64), generator=g, device=dev).argsort(-1) < 32, 1, -1)
        return x, up * sign[0]

    (xq, gq), (xk, gk) = rows(H), rows(Hk)
    w, b = torch.ones(64, device=dev), torch.zeros(64, device=dev)
    for norm in ("layer", "rms"):
        cfg = s3r.QKNormConfig(norm=norm, rope="none", eps=0.0)
        kw = dict(q_weight=w, k_weight=w, **(dict(q_bias=b, k_bias=b) if norm == "layer" else {}))
        got = s3r.qk_norm_rope_bwd(cfg, xq.to(dtype), xk.to(dtype), None, gq.to(dtype), gk.to(dtype), **kw)
        for n, x, up in (("q", xq, gq), ("k", xk, gk)):
            # a term is off by 2^-22; a thread adds at most 32 rows here (two tokens of 16 heads: 148 blocks
            # of 32 groups share 5,001), a block ten sums more, each rounded to fp32
            err = (2.0 ** -22 + 42 * 2.0 ** -24) * up.abs().sum((0, 1)).double()
            assert err.max() < 0.5
            assert ((getattr(got, n + "_weight").double() - (x * up).sum((0, 1))).abs() <= err).all()
            if norm == "layer":
                assert torch.equal(getattr(got, n + "_bias").long(), up.sum((0, 1)))


def case(dev, L, H, Hk, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    w = dict(q_weight=1 + 0.1 * r(64), q_bias=r(64), k_weight=1 + 0.1 * r(64), k_bias=r(64))
    pos = torch.randint(0, 500, (L, 2), generator=g, device=dev, dtype=torch.int32)
    q, gq, k, gk = r(L, H, 64), r(L, H, 64), r(L, Hk, 64), r(L, Hk, 64)
    return [t.to(dtype) for t in (q, k)], pos, [t.to(dtype) for t in (gq, gk)], w


CFG = s3r.QKNormConfig()


def both(c):
    x, pos, up, w = c
    return (*s3r.qk_norm_rope(CFG, *x, pos, **w), *s3r.qk_norm_rope_bwd(CFG, *x, pos, *up, **w))


@pytest.mark.parametrize("L,H,Hk", [(1, 16, 16), (700, 6, 3), (40000, 2, 1)])
def test_equal_calls_give_equal_bits(dev, L, H, Hk):
    c = case(dev, L, H, Hk, 11)
    first = both(c)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, both(c)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L,H,Hk", [(3, 16, 1), (700, 6, 3), (20000, 3, 2)])
def test_gradients_over_the_inputs_and_outputs_over_them(dev, L, H, Hk, dtype):
    (q, k), pos, up, w = case(dev, L, H, Hk, 12, dtype)
    want = s3r.qk_norm_rope_bwd(CFG, q, k, pos, *up, **w)
    x = q.clone(), k.clone()
    got = s3r.qk_norm_rope_bwd(CFG, *x, pos, *up, **w, grads=x)
    assert got.q is x[0] and all(torch.equal(a, b) for a, b in zip(want, got))
    want = s3r.qk_norm_rope(CFG, q, k, pos, **w)
    x = q.clone(), k.clone()
    got = s3r.qk_norm_rope(CFG, *x, pos, **w, out=x)
    assert got[0] is x[0] and all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_at_once(dev):
    cases = [case(dev, 3000, 4, 2, 13 + i) for i in range(2)]
    want = [both(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(both(cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


def test_captured_calls_replay_with_new_contents(dev):
    graphs = []
    for seed in (21, 22):
        c = case(dev, 500, 4, 2, seed)
        both(c)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = both(c)
        graphs.append((graph, c, res))
    for turn in range(2):
        for graph, c, _ in graphs:
            y = case(dev, 500, 4, 2, 30 + turn)
            for a, b in zip((*c[0], c[1], *c[2], *c[3].values()), (*y[0], y[1], *y[2], *y[3].values())):
                a.copy_(b)
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, c, res in graphs:
            assert all(torch.equal(a, b) for a, b in zip(res, both(c)))
