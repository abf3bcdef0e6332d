"""The selective scan's gradients against differences of the forward call on the GPU.

With f(s) = <y, dy> + <hT, dhT> of the fp32 forward call at inputs moved by s u, the slope along u is taken from
(8 (f(h) - f(-h)) - (f(2h) - f(-2h))) / 12h.  x, B, C, D and the initial state enter linearly: h = 1.  dt, A and the bias:
h = 2^-5, whose error, h^4 / 30 of a fifth derivative, is below 2^-14 of the slope's terms (5e-5 at most in fp64).  The
forward call's errors are held below 2^-17 of its outputs' root mean square elsewhere, and dy and dhT are drawn without
regard to them: f is off by a number of standard deviation 2^-17 (|y| + |hT|) (vectors' lengths) or less, the slope by
1.5 / h times that, and eight deviations are allowed.  The gradients are those of
fp32 inputs, or of the same values in bf16, whose 16-bit gradients are each off by 2^-8 of themselves at most.  They
are taken along themselves, where a slope is largest against those errors, and along a direction of random signs."""
import pytest
import torch

from test_gpu_ssm import backward, bf, f32, forward, make

pytestmark = pytest.mark.gpu
NAMES = ("x", "dt", "A", "B", "C", "D", "bias", "h0")
LINEAR = ("x", "B", "C", "D", "h0")


def value(d):
    y, hT = forward(d)
    dot = lambda a, b: (a.double() * b.double()).sum().item()                              # noqa: E731
    size = lambda t: t.double().pow(2).sum().sqrt().item()                                 # noqa: E731
    return dot(y, d["dy"]) + dot(hT, d["dhT"]), size(y) + size(hT)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv,hg,T", [(64, 64, (2, 1), 150), (128, 128, (2, 2), 70), (128, 64, (3, 1), 1100)])
def test_slopes(dtype, dk, dv, hg, T):
    d = make(f32, [T], *hg, dk, dv, packed=False, state=True, seed=12, wide=False)
    for k in ("x", "B", "C", "dt", "dy"):              # values that 16 bits hold
        d[k] = d[k].to(bf).float().contiguous()
    e = {k: t.to(dtype) if k in ("x", "B", "C", "dt", "dy") else t for k, t in d.items()}
    got = dict(zip(NAMES, backward(e)))
    g = torch.Generator().manual_seed(13)
    for k in NAMES:
        grad = got[k].double()
        h = 1.0 if k in LINEAR else 2.0 ** -5
        along = grad / grad.pow(2).mean().sqrt()
        signs = torch.randint(0, 2, d[k].shape, generator=g).double().to(grad.device) * 2 - 1
        for u, tells in ((along.clamp(-4, 4).to(f32).double(), True), (signs, False)):
            f, noise = zip(*[value({**d, k: (d[k].double() + s * h * u).to(f32)}) for s in (1, -1, 2, -2)])
            slope = (8 * (f[0] - f[1]) - (f[2] - f[3])) / (12 * h)
            have, terms = (grad * u).sum().item(), (grad * u).abs().sum().item()
            # (moved inputs are rounded to fp32: 2^-24 of themselves, far below the rest)
            allowed = 8 * 2.0 ** -17 * max(noise) * 1.5 / h + (2.0 ** -13 + (2.0 ** -8 if got[k].dtype == bf else 0)) * terms
            assert abs(have - slope) <= allowed, (k, have, slope, allowed)
            assert not tells or allowed < abs(have) / 16, (k, have, allowed)
