"""The fp64 reference of the scan's gradients against automatic differentiation and against differences of the
recurrence (CPU)."""
import torch

import ssm_ref as R


def _case(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    H, G, dk, dv = 4, 2, 3, 5
    cu = [0, 4, 4, 11]
    d = dict(x=r(1, 11, H, dv), dt=r(1, 11, H), A=-torch.rand(H, generator=g, dtype=torch.float64) * 2, B=r(1, 11, G, dk),
             C=r(1, 11, G, dk), D=r(H), bias=r(H), h0=r(3, H, dk, dv), cu=cu)
    return d, r(1, 11, H, dv), r(3, H, dk, dv)


def test_formulas_against_autograd():
    d, dy, dhT = _case()
    ref = R.scan_grads(dy=dy, dhT=dhT, **d)
    names = ("x", "dt", "A", "B", "C", "D", "bias", "h0")
    leaves = [d[k].clone().requires_grad_() for k in names]
    y, hT = R.scan(**dict(zip(names, leaves)), cu=d["cu"])
    grads = torch.autograd.grad((y * dy).sum() + (hT * dhT).sum(), leaves)
    for k, got in zip(names, grads):
        assert torch.allclose(got, ref["d" + k], rtol=1e-10, atol=1e-12), k


def test_formulas_against_differences():
    d, dy, dhT = _case(1)
    ref = R.scan_grads(dy=dy, dhT=dhT, **d)

    def loss(**over):
        y, hT = R.scan(**{**d, **over})
        return ((y * dy).sum() + (hT * dhT).sum()).item()

    g = torch.Generator().manual_seed(7)
    for k in ("x", "dt", "A", "B", "C", "D", "bias", "h0"):
        v = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        eps = 1e-6
        diff = (loss(**{k: d[k] + eps * v}) - loss(**{k: d[k] - eps * v})) / (2 * eps)
        want = (ref["d" + k] * v).sum().item()
        # central differences: curvature eps^2 and rounding 2^-53 / eps of terms of size about 1e3
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want)), (k, diff, want)


def test_conv_grads_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, w, b, h0, dy, dhT = r(1, 9, 3), r(3, 4), r(3), r(3, 3, 3), r(1, 9, 3), r(3, 3, 3)
    cu = [0, 2, 2, 9]
    grads = R.conv_grads(x, w, dy, b, h0, dhT, cu)

    def loss(x, w, b, h0):
        y, hT = R.conv(x, w, b, h0, cu)
        return ((y * dy).sum() + (hT * dhT).sum()).item()

    args = [x, w, b, h0]
    for i in range(4):
        v, eps = r(*args[i].shape), 1e-6
        up = [a + eps * v if j == i else a for j, a in enumerate(args)]
        dn = [a - eps * v if j == i else a for j, a in enumerate(args)]
        diff, want = (loss(*up) - loss(*dn)) / (2 * eps), (grads[i] * v).sum().item()
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want))
