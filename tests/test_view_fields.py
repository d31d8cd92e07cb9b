"""Config values at and beyond the range of the library's 32-bit fields (include/s3r_view.h): what reaches
the library is the value, or the call is refused."""
import pytest

import sparse_global_attention_s3r_b200 as s3r


def fields(nseg=1, Lq=1000, Lk=2000, **kw):
    return s3r.ViewConfig(H=2, **kw)._params(Lq, Lk, nseg, True, None, (0,) * 12)


@pytest.mark.parametrize("most,got", [(None, 1000), (0, 0), (7, 7), (1000, 1000), (1001, 1000),
                                      (2 ** 31 - 1, 1000), (2 ** 31, 1000), (2 ** 32, 1000),
                                      (2 ** 32 + 5, 1000), (2 ** 64 + 5, 1000), (-1, -1),
                                      (-2 ** 32 + 400, -1)])
def test_bounds_on_a_segment(most, got):
    assert fields(max_q=most).max_q == got
    assert fields(Lk=1000, max_k=most).max_k == got


@pytest.mark.parametrize("scale", [1e-46, 1e-300, 1e39, 1e300])
def test_scale_that_fp32_does_not_hold_is_refused(scale):
    with pytest.raises(ValueError, match="scale must be positive"):
        fields(scale=scale)


@pytest.mark.parametrize("scale", [1e-45, 1e-38, 0.125, 3e38])
def test_scale_that_fp32_holds_is_taken(scale):
    assert 0 < fields(scale=scale).scale < float("inf")


def test_more_segments_than_the_field_holds_are_refused():
    assert fields(nseg=2 ** 31 - 1).nseg == 2 ** 31 - 1
    for n in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="segments"):
            fields(nseg=n)
