"""The selective scan's gradients of dt, element by element: against fp64, within the roundings of what a token's ddt is
added up from inside its chunk (64 tokens, fp32 32), and not of what all later tokens of a sequence add up to.

Tolerance.  All that goes into ddt is fp32 whatever the inputs' type (16-bit inputs enter products exactly, states as
three terms).  A term is the product of two dot products of up to 128 channels and of a decay from at most three
factors; 64 terms are added up, and the states hold up to 2^9 tokens that still weigh: below 2^10 roundings of 2^-24 each,
of either sign, which add up like the root of their number, 2^-19 of the magnitudes; four times that for one entry
among thousands, and as much again for what the MFMAs drop towards minus infinity (2^10 times 2^-25 of partial sums, which
with inputs of either sign are an eighth of the magnitudes or less): 2^-16.  An output in bf16 adds its rounding."""
import pytest
import torch

import ssm_ref as R
import ssm_ways as W
from kda_testutil import say
from test_gpu_ssm import SIZES, backward, bf, f32, make

pytestmark = pytest.mark.gpu
BATCHES = [([1290], False, (3, 1)), ([1100, 0, 1, 513, 64], True, (4, 2)), ([512, 1024, 600], True, (3, 3)), ([200, 200], False, (6, 1))]


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("lens,packed,hg", BATCHES)
def test_ddt(dtype, dk, dv, lens, packed, hg):
    d = make(dtype, lens, *hg, dk, dv, packed=packed, state=True, scale_dt=2.0)
    got = backward(d)[1]
    torch.cuda.synchronize()
    args = dict(d["ref"], dy=R.f64(d["dy"]), dhT=R.f64(d["dhT"]), chunk=64 if dtype == bf else 32)
    ref, mag = W.ddt(**args), W.ddt(**args, magnitude=True)
    beyond = ((got.double().cpu() - ref).abs() - torch.finfo(dtype).eps / 2 * ref.abs()) / mag.clamp(min=1e-300)
    say(f"  ddt: {beyond.max().item():.2e} of the magnitudes")
    assert beyond.max().item() <= 2.0 ** -16
