"""The package is imported where torch was built without CUDA: host helpers and refusals work there."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
import torch.cuda
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):  # what such a build does not have
    delattr(torch._C, n)
import sparse_global_attention_s3r_b200 as s3r
assert s3r.view_positions(1, 1, 2).tolist() == [[1, 1], [1, 2]]
x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
for call in (lambda: s3r.qk_norm_rope(s3r.QKNormConfig(rope="none"), x, x),
             lambda: s3r.view_attn_fwd(s3r.ViewConfig(H=2), x, x, x, *[torch.zeros(2, dtype=torch.int32)] * 2)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("not refused")
"""


def test_import_where_torch_has_no_cuda():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
