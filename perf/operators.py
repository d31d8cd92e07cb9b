"""Cases of the dense operators around the sparse global attention: the per-head norm of queries and
keys with the position rotation, and the dense attention inside views (or a scene, or against a
cache of earlier views), each forward and backward.

`run` computes a case in plain torch operations, or, where `own` is true, through the package's
entry points. The operators, on rows of 64 channels per (token, head):

  qk_norm_rope   x -> R(pos) (norm(x) * weight + bias), for queries and keys in one call. norm is
                 the layer norm or the root-mean-square norm over the 64 channels. R rotates the
                 channel pairs (i, i + 32) by pos * base^(-i/32) ("1d"), or the pairs (i, i + 16)
                 of each half by y * base^(-i/16) (first half) and x * base^(-i/16) ("2d").
  view_attn      out = softmax(scale q k^T) v of every query over the keys of its own segment;
                 segment s holds queries q_offs[s] .. q_offs[s+1] and keys k_offs[s] .. k_offs[s+1].
                 A segment without keys gives zeros and lse = -inf, and so do rows past the last
                 segment. Heads h of q share key head h // (H / Hkv).
"""
import random

import torch

own = False

D = 64
SCALE = 0.125  # 1 / sqrt(64)
BASE = {"1d": 10000.0, "2d": 100.0}
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    """Token geometry of the repository's workloads: views of 1,374 tokens (5 special + 37 x 37
    patches), 16 heads."""
    def rope(name, bwd, L, H, Hk, dtype, norm, rot, views):
        return dict(name=name, op="rope", bwd=bwd, L=L, H=H, Hk=Hk, dtype=dtype, norm=norm, rot=rot,
                    views=views)

    def attn(name, bwd, n, q, k, H, Hkv, ragged, tail):
        return dict(name=name, op="attn", bwd=bwd, n=n, q=q, k=k, H=H, Hkv=Hkv, ragged=ragged, tail=tail)

    return [
        # one token appended to a long stream: only latency counts
        rope("rope_one_token", False, 1, 16, 16, "bf16", "rms", "1d", False),
        # the queries and keys of a 100-view layer, out of one packed projection
        rope("rope_100_views", False, 137400, 16, 16, "bf16", "layer", "2d", True),
        # a training step at 32 views: gradients of the projection and of the norms' weights
        rope("rope_grad_32_views", True, 43968, 16, 16, "bf16", "layer", "2d", True),
        # fp32 activations, an odd token count, fewer key heads, far positions
        rope("rope_grad_odd_f32", True, 5497, 6, 3, "f32", "rms", "1d", False),
        # attention inside each of 32 views
        attn("attn_32_views", False, 32, 1374, 1374, 16, 16, 0, 0),
        # every token of 8 views with every other: the dense layer the sparse one stands for
        attn("attn_scene_8_views", False, 1, 10992, 10992, 16, 16, 0, 0),
        # one query token over the cached keys of 100 views
        attn("attn_token_cache", False, 1, 1, 137400, 16, 16, 0, 0),
        # views of unequal token counts, some empty, keys shared by four heads, rows left over
        attn("attn_ragged", False, 48, 1374, 1374, 16, 4, 7, 37),
        # the gradients of the three layouts above, and of a small layer
        attn("attn_grad_32_views", True, 32, 1374, 1374, 16, 16, 0, 0),
        attn("attn_grad_scene_8_views", True, 1, 10992, 10992, 16, 16, 0, 0),
        attn("attn_grad_ragged", True, 48, 1374, 1374, 16, 4, 8, 37),
        attn("attn_grad_small", True, 4, 256, 256, 2, 2, 0, 0),
    ]


def _log(rng, lo, hi):
    """An integer of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    if rng.random() < 0.35:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        bwd = rng.random() < 0.5
        Hk = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        H = Hk * rng.choice([1, 1, 1, 2, 4]) if Hk <= 4 else Hk
        most = 137400 * 32 * 2 // ((H + Hk) * (4 if dtype == "f32" else 2) * (2 if bwd else 1))
        return dict(op="rope", bwd=bwd, L=_log(rng, 1, most), H=H, Hk=Hk, dtype=dtype,
                    norm=rng.choice(["layer", "rms"]), rot=rng.choice(["1d", "2d"]), views=False)
    bwd = rng.random() < 0.5
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    H = Hkv * rng.choice([1, 1, 2, 4]) if Hkv <= 4 else Hkv
    n = _log(rng, 1, 48)
    most = 16 * 10992 * 10992 // (H * n)  # query-key pairs of one segment and head
    q = _log(rng, 1, min(10992, most))
    k = q if rng.random() < 0.5 else _log(rng, 1, min(137400 // n, max(1, most // q)))
    k = min(k, max(1, most // q))
    if bwd:  # one key alone has P = 1 and dq = dk = 0: nothing to compare
        k = max(k, 16)
    return dict(op="attn", bwd=bwd, n=n, q=q, k=k, H=H, Hkv=Hkv,
                ragged=rng.choice([0, rng.randrange(1, 1 << 20)]), tail=rng.choice([0, rng.randrange(1, 300)]))


def _lengths(case):
    """Queries and keys of each segment: the full counts, or spread below them with some at zero."""
    n, q, k = case["n"], case["q"], case["k"]
    if not case["ragged"]:
        return [q] * n, [k] * n
    r = random.Random(case["ragged"])

    def some(top):
        return [0 if r.random() < 0.08 else r.randint(1, top) for _ in range(n)]

    lq = some(q)
    lk = list(lq) if q == k else some(k)
    if q == k and n > 1:  # a view that lost its keys, and one that lost its queries
        lk[r.randrange(n)] = 0
        lq[r.randrange(n)] = 0
    lq[0], lk[0] = q, k  # one is whole
    return lq, lk


def _offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def work(case):
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        rows = case["L"] * (case["H"] + case["Hk"])
        pos = case["L"] * (8 if case["rot"] == "2d" else 4)
        return {"bytes": rows * D * size * (3 if case["bwd"] else 2) + pos,
                "flops": rows * D * (24 if case["bwd"] else 12)}
    lq, lk = _lengths(case)
    H, Hkv = case["H"], case["Hkv"]
    q = (sum(lq) + case["tail"]) * H * D * 2
    kv = (sum(lk) + case["tail"]) * Hkv * D * 2
    lse = (sum(lq) + case["tail"]) * H * 4
    pairs = sum(a * b for a, b in zip(lq, lk)) * H
    if case["bwd"]:  # q, out, dout read, dq written; k, v read, dk, dv written
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * D * pairs}
    return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * D * pairs}


def _randn(shape, g, dtype=torch.bfloat16, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        L, H, Hk, dtype = case["L"], case["H"], case["Hk"], TYPES[case["dtype"]]
        x = _randn((L, H + Hk, D), g, dtype)  # queries and keys of one projection
        s["q"], s["k"] = x[:, :H], x[:, H:]
        layer = case["norm"] == "layer"
        for n in "qk":
            s[n + "_weight"] = 1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")
            s[n + "_bias"] = 0.1 * torch.randn(D, generator=g, device="cuda") if layer else None
        if case["views"]:  # (y, x) of 37 x 37 patches, counted from 1; special tokens at 0
            t = torch.arange(L, device="cuda") % 1374 - 5
            pos = torch.stack([t // 37 + 1, t % 37 + 1], 1)
            s["pos"] = torch.where(t[:, None] < 0, 0, pos).to(torch.int32)
        elif case["rot"] == "2d":
            s["pos"] = torch.randint(0, 512, (L, 2), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["pos"] = (torch.randint(0, 1 << 20, (1,), generator=g, device="cuda", dtype=torch.int32)
                        + torch.arange(L, device="cuda", dtype=torch.int32))
        if case["bwd"]:
            s["dq_out"], s["dk_out"] = _randn((L, H, D), g, dtype, 0.01), _randn((L, Hk, D), g, dtype, 0.01)
    else:
        lq, lk = _lengths(case)
        s["q_offs"] = torch.tensor(_offsets(lq), dtype=torch.int32, device="cuda")
        s["k_offs"] = torch.tensor(_offsets(lk), dtype=torch.int32, device="cuda")
        s["max_q"], s["max_k"] = max(max(lq), 1), max(max(lk), 1)
        Lq, Lk = max(1, sum(lq) + case["tail"]), max(1, sum(lk) + case["tail"])
        # normed queries and keys: logits of a standard deviation near 1.5
        s["q"], s["k"], s["v"] = (_randn((Lq, case["H"], D), g, gain=1.5), _randn((Lk, case["Hkv"], D), g),
                                  _randn((Lk, case["Hkv"], D), g))
        if case["bwd"]:
            s["dout"] = _randn((Lq, case["H"], D), g, gain=0.01)
            s["out"], s["lse"] = _plain_attn(s)  # what the forward left
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _angles(pos, rot):
    """cos and sin [L, 1, 32] of the 32 rotated pairs, from angles in 64 bits."""
    p = pos.double()
    if rot == "1d":
        f = BASE[rot] ** (-torch.arange(32, device=p.device, dtype=torch.float64) / 32)
        a = p[:, None] * f
    else:
        f = BASE[rot] ** (-torch.arange(16, device=p.device, dtype=torch.float64) / 16)
        a = torch.cat([p[:, :1] * f, p[:, 1:] * f], 1)
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _pairs(x, rot):
    """The first and the second channel of each rotated pair, [L, H, 32] each."""
    if rot == "1d":
        return x[..., :32], x[..., 32:]
    y = x.reshape(*x.shape[:-1], 2, 2, 16)
    return y[..., 0, :].flatten(-2), y[..., 1, :].flatten(-2)


def _unpair(a, b, rot):
    if rot == "1d":
        return torch.cat([a, b], -1)
    a, b = a.unflatten(-1, (2, 16)), b.unflatten(-1, (2, 16))
    return torch.stack([a, b], -2).flatten(-3)


def _normed(x, norm):
    x = x.float()
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def _plain_rope(x, weight, bias, cos, sin, case):
    y = _normed(x, case["norm"])[0] * weight
    if bias is not None:
        y = y + bias
    a, b = _pairs(y, case["rot"])
    return _unpair(a * cos - b * sin, b * cos + a * sin, case["rot"]).to(x.dtype)


def _plain_rope_grad(x, weight, bias, cos, sin, dout, case):
    a, b = _pairs(dout.float(), case["rot"])
    dy = _unpair(a * cos + b * sin, b * cos - a * sin, case["rot"])
    xhat, rstd = _normed(x, case["norm"])
    dweight = (dy * xhat).sum((0, 1), dtype=torch.float64).float()
    dbias = dy.sum((0, 1), dtype=torch.float64).float() if bias is not None else None
    dh = dy * weight
    dx = dh - xhat * (dh * xhat).mean(-1, keepdim=True)
    if case["norm"] == "layer":
        dx = dx - dh.mean(-1, keepdim=True)
    return (dx * rstd).to(x.dtype), dweight, dbias


def _rows(offs, most, total):
    """Row numbers [n, most] of each segment, those past its end at `total`, and the same as truth
    values of what is inside."""
    i = torch.arange(most, device=offs.device)
    inside = i < (offs[1:] - offs[:-1])[:, None]
    return torch.where(inside, offs[:-1, None] + i, total), inside


def _padded(x, rows, heads):
    """[n, heads, most, 64] in 32 bits, rows past a segment's end at zero."""
    x = torch.cat([x, x.new_zeros((1, *x.shape[1:]))]).float()[rows]
    if x.shape[2] != heads:
        x = x.repeat_interleave(heads // x.shape[2], 2)
    return x.transpose(1, 2)


def _softmax(q, k, keys):
    logits = (q @ k.transpose(-1, -2)) * SCALE
    logits.masked_fill_(~keys[:, None, None], -torch.inf)
    top = logits.amax(-1, keepdim=True).clamp_min(-1e30)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)  # -inf where there are no keys
    return p.div_(torch.where(total > 0, total, 1.0)), lse


def _back(x, rows, total, width, fill=0.0):
    """[n, heads, most, ...] to [total, heads, ...], rows of no segment at `fill`."""
    out = torch.full((total + 1, x.shape[1], *width), fill, dtype=torch.float32, device=x.device)
    out[rows] = x.transpose(1, 2)
    return out[:total]


def _plain_attn(s):
    q, k, v = s["q"], s["k"], s["v"]
    qr, _ = _rows(s["q_offs"], s["max_q"], q.shape[0])
    kr, keys = _rows(s["k_offs"], s["max_k"], k.shape[0])
    H = q.shape[1]
    p, lse = _softmax(_padded(q, qr, H), _padded(k, kr, H), keys)
    out = _back(p @ _padded(v, kr, H), qr, q.shape[0], (D,))
    lse = _back(lse, qr, q.shape[0], (), -torch.inf)
    return out.to(q.dtype), lse.t().contiguous()


def _plain_attn_grad(s):
    q, k, v = s["q"], s["k"], s["v"]
    Lq, Lk, H, Hkv = q.shape[0], k.shape[0], q.shape[1], k.shape[1]
    qr, _ = _rows(s["q_offs"], s["max_q"], Lq)
    kr, keys = _rows(s["k_offs"], s["max_k"], Lk)
    qp, kp, vp, do = (_padded(q, qr, H), _padded(k, kr, H), _padded(v, kr, H), _padded(s["dout"], qr, H))
    p, _ = _softmax(qp, kp, keys)
    dv = p.transpose(-1, -2) @ do
    ds = do @ vp.transpose(-1, -2)
    ds = ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p).mul_(SCALE)
    del p
    dq, dk = ds @ kp, ds.transpose(-1, -2) @ qp
    dk, dv = (x.unflatten(1, (Hkv, H // Hkv)).sum(2) for x in (dk, dv))
    return (_back(dq, qr, Lq, (D,)).to(q.dtype), _back(dk, kr, Lk, (D,)).to(q.dtype),
            _back(dv, kr, Lk, (D,)).to(q.dtype))


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "attn":
        return _plain_attn_grad(s) if case["bwd"] else _plain_attn(s)
    cos, sin = _angles(s["pos"], case["rot"])
    f = (lambda n: _plain_rope_grad(s[n], s[n + "_weight"], s[n + "_bias"], cos, sin, s["d" + n + "_out"], case)) \
        if case["bwd"] else (lambda n: _plain_rope(s[n], s[n + "_weight"], s[n + "_bias"], cos, sin, case))
    return f("q"), f("k")


def _own(s, case):
    import sparse_global_attention_s3r_b200 as s3r

    if case["op"] == "attn":
        cfg = s3r.ViewConfig(H=case["H"], Hkv=case["Hkv"], max_q=s["max_q"], max_k=s["max_k"])
        offs = s["q_offs"], s["k_offs"]
        if case["bwd"]:
            return s3r.view_attn_bwd(cfg, s["q"], s["k"], s["v"], *offs, s["out"], s["lse"], s["dout"])
        return s3r.view_attn_fwd(cfg, s["q"], s["k"], s["v"], *offs)
    cfg = s3r.QKNormConfig(norm=case["norm"], rope=case["rot"], base=BASE[case["rot"]], eps=EPS)
    weights = dict(q_weight=s["q_weight"], q_bias=s["q_bias"], k_weight=s["k_weight"], k_bias=s["k_bias"])
    if case["bwd"]:
        g = s3r.qk_norm_rope_bwd(cfg, s["q"], s["k"], s["pos"], s["dq_out"], s["dk_out"], **weights)
        return (g.q, g.q_weight, g.q_bias), (g.k, g.k_weight, g.k_bias)
    return s3r.qk_norm_rope(cfg, s["q"], s["k"], s["pos"], **weights)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, one head (and segment) at a time
# ---------------------------------------------------------------------------------------------
def _exact_rope(s, case, n):
    x, w, b = s[n].double(), s[n + "_weight"].double(), s[n + "_bias"]
    pos, rot = s["pos"].double(), case["rot"]
    c = torch.arange(D, device=x.device)
    if rot == "1d":
        partner, first = (c + 32) % 64, c < 32
        angle = pos[:, None] * torch.pow(BASE[rot], -(c % 32).double() / 32)
    else:
        partner, first = c ^ 16, (c & 16) == 0
        axis = pos[:, (c >= 32).long()]
        angle = axis * torch.pow(BASE[rot], -(c % 16).double() / 16)
    sign = torch.where(first, -1.0, 1.0).double()
    cos, sin = angle.cos(), angle.sin() * sign
    centre = x.mean(-1, keepdim=True) if case["norm"] == "layer" else 0.0
    sigma = ((x - centre) ** 2).mean(-1, keepdim=True).add(EPS).sqrt()
    xhat = (x - centre) / sigma
    if not case["bwd"]:
        y = xhat * w + (b.double() if b is not None else 0.0)
        return y * cos[:, None] + y[..., partner] * sin[:, None]
    g = s["d" + n + "_out"].double()
    # channel c of y reaches output c by cos and output partner(c) by that output's sin
    dy = g * cos[:, None] + (g * sin[:, None])[..., partner]
    dw, db = (dy * xhat).sum((0, 1)), dy.sum((0, 1)) if b is not None else None
    h = dy * w
    # the Jacobian of xhat: (I - 1 1^T/64 - xhat xhat^T/64) / sigma
    dx = (h - xhat * (h * xhat).sum(-1, keepdim=True) / D
          - (h.sum(-1, keepdim=True) / D if case["norm"] == "layer" else 0.0)) / sigma
    return dx, dw, db


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case, "q"), _exact_rope(s, case, "k")
    q, k, v = s["q"], s["k"], s["v"]
    H, group = case["H"], case["H"] // case["Hkv"]
    qo, ko = s["q_offs"].tolist(), s["k_offs"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((H, q.shape[0]), -torch.inf, dtype=torch.float64, device=q.device)
    dk, dv = (torch.zeros(k.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    for i in range(case["n"]):
        for h in range(H):
            a, b = slice(qo[i], qo[i + 1]), slice(ko[i], ko[i + 1])
            qs, ks, vs = q[a, h].double(), k[b, h // group].double(), v[b, h // group].double()
            if qs.shape[0] == 0 or ks.shape[0] == 0:
                continue
            t = qs.mm(ks.t()) * SCALE
            z = torch.logsumexp(t, 1, keepdim=True)
            p = torch.exp(t - z)
            if not case["bwd"]:
                out[a, h], lse[h, a] = p.mm(vs), z[:, 0]
                continue
            go = s["dout"][a, h].double()
            o = p.mm(vs)
            dt = p * (go.mm(vs.t()) - (go * o).sum(1, keepdim=True))
            out[a, h] = dt.mm(ks) * SCALE  # dq
            dk[b, h // group] += dt.t().mm(qs) * SCALE
            dv[b, h // group] += p.t().mm(go)
    return (out, dk, dv) if case["bwd"] else (out, lse)
