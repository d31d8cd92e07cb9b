"""Dense attention of many segments of which nearly all are empty: the warps that wait for an item's tiles
must not take a long run of items without rows for a lost one."""
import pytest
import torch

import sparse_global_attention_s3r_b200 as s3r

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def test_seven_hundred_million_items_without_rows(dev):
    """65,535 heads by 11,000 segments, of which the first and the last hold one token each: about 2.3 s of
    items without rows in each kernel, longer than one wait may take."""
    H, n = 65535, 11000
    g = torch.Generator(device=dev).manual_seed(80)
    q, k, v, dout = (torch.randn((2, H, 64), generator=g, device=dev).to(torch.bfloat16) for _ in range(4))
    dout = (dout.float() * 0.1).to(torch.bfloat16)
    offs = torch.ones(n + 1, dtype=torch.int32, device=dev)
    offs[0], offs[-1] = 0, 2
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    cfg = s3r.ViewConfig(H=H, max_q=1, max_k=1)
    out, lse = s3r.view_attn_fwd(cfg, q, k, v, offs, offs, dev_status=word)
    assert s3r.read_device_status(word) == 0
    # one key: P is 1 within 2^-20, which is below a half step of bf16 around any v
    assert ((out.double() - v.double()).abs() <= 2.0 ** -8 * v.double().abs()).all()
    want = (q.double() * k.double()).sum(-1).t() / 8
    assert ((lse.double() - want).abs() <= 1e-5 * (1 + want.abs())).all()
    dq, dk, dv = s3r.view_attn_bwd(cfg, q, k, v, offs, offs, out, lse, dout, dev_status=word)
    assert s3r.read_device_status(word) == 0
    assert ((dv.double() - dout.double()).abs() <= 2.0 ** -8 * dout.double().abs()).all()
    # dS = P dP (1 - P): at most 2^-15 of |dP| (at most 64 terms of at most 0.6 * 6), times 6 / 8
    assert max(dq.abs().max(), dk.abs().max()) <= 2.0 ** -15 * 64 * 3.6 * 0.75
