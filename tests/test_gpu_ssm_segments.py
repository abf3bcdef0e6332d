"""Sequences in several segments at every head size, forward and backward, with several heads a group and several groups:
the eight-wave passes of d_v = 128 among them.  Tolerances are those of test_gpu_ssm."""
import pytest

from test_gpu_ssm import SIZES, bf, check_backward, check_forward, f32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("lens,packed,hg", [([1300], False, (6, 2)), ([1100, 0, 1, 1537, 64], True, (4, 2)), ([2100, 2100], False, (3, 1)),
                                            ([1030], True, (2, 2))])
def test_segments(dtype, dk, dv, lens, packed, hg):
    d = make(dtype, lens, *hg, dk, dv, packed=packed, state=True, scale_dt=2.0, seed=21)
    check_forward(d, dtype)
    check_backward(d, dtype)
