"""Which shapes of the GPU tests have the dense attention's walks split into pieces: the tests that are about
split walks have to stay so when the estimates behind the number of pieces change."""
import ctypes

import pytest

import sparse_global_attention_s3r_b200 as s3r
from sparse_global_attention_s3r_b200 import _lib


def workspaces(Lq, Lk, H, nseg, max_q, max_k):
    p = ctypes.byref(s3r.ViewConfig(H=H, max_q=max_q, max_k=max_k)._params(Lq, Lk, nseg, True, None, (0,) * 12))
    lib = _lib.load()
    d = max(256, -(-Lq * H * 4 // 256) * 256)
    return lib.s3r_view_attn_workspace_bytes(p), lib.s3r_view_attn_bwd_workspace_bytes(p) - d


@pytest.mark.parametrize("shape", [
    (3, 9000, 1, 1, 3, 9000),            # one long segment
    (100, 2060, 1, 2, None, None),       # unusable offsets
    (43, 4900, 1, 2, 64, 4900),          # captured graphs
    (300000, 300000, 2, 2, 30, 2300),    # few rows of large tensors
    (120, 6001, 1, 3, 50, 2001),         # an unusable segment between two others
    (1, 5000, 1, 1, None, None),         # workspaces that do not fit
])
def test_shapes_that_are_split(shape):
    fwd, bwd = workspaces(*shape)
    assert fwd > 0 and bwd > 0


@pytest.mark.parametrize("shape", [(1374, 1374, 16, 1, None, None), (120, 1801, 1, 3, 50, 601)])
def test_shapes_that_are_not_split(shape):
    assert workspaces(*shape)[0] == 0
