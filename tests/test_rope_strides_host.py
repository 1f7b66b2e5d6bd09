"""Strides of the gradients of norm and rotation, without a GPU: what lies like its input is taken, whatever torch calls
the step of a dimension that never steps."""
import pytest
import torch

from tests.test_cache_host import _Fake, bpa, streams  # noqa: F401


def call(bpa, q, dq):  # noqa: F811
    dy, ws = _Fake(torch.zeros(q.shape)), _Fake(torch.zeros(4096, dtype=torch.uint8))
    return bpa.bpa_rope_bwd(_Fake(q), None, dy, None, dq=_Fake(dq), workspace_buf=ws)


BUF = torch.zeros(4096)


@pytest.mark.parametrize("shape,a,b", [((1, 5, 4, 8), (160, 32, 8, 1), (7, 32, 8, 1)), ((2, 1, 4, 8), (32, 32, 8, 1), (32, 99, 8, 1)),
                                       ((2, 5, 1, 8), (40, 8, 8, 1), (40, 8, 3, 1)), ((1, 4, 8), (32, 8, 1), (5, 8, 1)),
                                       ((6, 1, 8), (8, 8, 1), (8, 1, 1)), ((1, 1, 1, 8), (8, 8, 8, 1), (0, 1, 2, 1))])
def test_steps_of_a_dimension_of_one_say_nothing(bpa, streams, shape, a, b):  # noqa: F811
    q, dq = BUF.as_strided(shape, a), BUF.as_strided(shape, b)
    got = call(bpa, q, dq)
    assert got[0].t is dq and streams[2] == [("bpa_rope_bwd", 0x10)]


@pytest.mark.parametrize("shape,a,b", [((2, 5, 4, 8), (160, 32, 8, 1), (320, 32, 8, 1)), ((1, 5, 4, 8), (160, 32, 8, 1), (160, 64, 8, 1)),
                                       ((1, 5, 2, 8), (160, 32, 8, 1), (160, 32, 16, 1)), ((6, 1, 8), (8, 8, 1), (16, 8, 1)),
                                       ((6, 2, 8), (16, 8, 1), (32, 16, 1))])
def test_other_strides_are_refused(bpa, streams, shape, a, b):  # noqa: F811
    with pytest.raises(ValueError, match="strides"):
        call(bpa, BUF.as_strided(shape, a), BUF.as_strided(shape, b))
    assert not streams[2]
