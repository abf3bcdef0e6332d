"""The selective scan's gradients of dt, formed in chunks from the ways between the tokens, in fp64 on the CPU: what the
kernels add up, and with the magnitudes of the inputs how large the terms of those sums are.

With c_i = A (delta_1 + .. + delta_i) inside a chunk, S the state before it and G the gradient of the one behind it,
    z_ij = e^(c_i - c_j) delta_j (C_i . B_j) (x_j . dy_i), j < i,   thr = e^c_n <G, S>,
    p_i = e^c_i dy_i . S^T C_i,   r_j = delta_j e^(c_n - c_j) x_j . G^T B_j,
    dg_t = thr + sum_{i >= t} (sum_j z_ij - sum_k z_ki + p_i) + sum_{j < t} r_j,
    x_t . u_t = sum_{i >= t} e^(c_i - c_t) (C_i . B_t) (x_t . dy_i) + r_t / delta_t,
    ddt_t = (x_t . u_t + A dg_t) / (1 + e^-(dt_t + bias))."""
from __future__ import annotations

import torch

import ssm_ref as R


def ddt(x, dt, A, B, C, dy, bias=None, h0=None, dhT=None, cu=None, D=None, chunk=64, magnitude=False):
    """ddt [B, T, H]; with `magnitude` the sums of the magnitudes of all that a token's ddt is added up from."""
    if magnitude:
        x, B, C, dy = x.abs(), B.abs(), C.abs(), dy.abs()
        h0, dhT = (None if t is None else t.abs() for t in (h0, dhT))
    nb, T, H, dv = x.shape
    dk = B.shape[-1]
    pre = dt if bias is None else dt + bias
    delta, slope = R.softplus(pre), torch.sigmoid(pre)
    Bh, Ch = R.heads(B, H), R.heads(C, H)
    out = torch.zeros_like(dt)
    for n, (b, lo, hi) in enumerate(R.spans(nb, T, cu)):
        cuts = [(a, min(a + chunk, hi)) for a in range(lo, hi, chunk)]
        zero = x.new_zeros(H, dk, dv)
        S, G = (zero if h0 is None else h0[n]), (zero if dhT is None else dhT[n])
        states = []
        for a, e in cuts:
            states.append(S)
            d = delta[b, a:e]
            c = d.cumsum(0) * A
            w = (torch.exp(c[-1] - c) * d)[..., None]
            S = S * torch.exp(c[-1])[:, None, None] + (w * Bh[b, a:e]).permute(1, 2, 0) @ x[b, a:e].transpose(0, 1)
        for (a, e), S in zip(reversed(cuts), reversed(states)):
            d, xs, ys = delta[b, a:e], x[b, a:e], dy[b, a:e]
            Bc, Cc = Bh[b, a:e], Ch[b, a:e]
            c = d.cumsum(0) * A                                              # [n, H]
            way = torch.exp((c[:, None] - c[None]).clamp(max=0)) * torch.ones(e - a, e - a, dtype=x.dtype).tril()[..., None]
            m = way * torch.einsum("ihk,jhk->ijh", Cc, Bc) * torch.einsum("ihv,jhv->ijh", ys, xs)
            z = m * d[None] * torch.ones(e - a, e - a, dtype=x.dtype).tril(-1)[..., None]
            before, after = torch.exp(c), torch.exp(c[-1] - c)
            p = before * torch.einsum("ihk,hkv,ihv->ih", Cc, S, ys)
            later = after * torch.einsum("ihk,hkv,ihv->ih", Bc, G, xs)       # r / delta
            thr = torch.exp(c[-1]) * (G * S).sum((-1, -2))
            ends = z.sum(0)
            zp = z.sum(1) + (ends if magnitude else -ends) + p
            r = d * later
            dg = thr + zp.flip(0).cumsum(0).flip(0) + r.cumsum(0) - r
            xu = m.sum(0) + later
            out[b, a:e] = (xu + (A.abs() if magnitude else A) * dg) * slope[b, a:e]
            G = G * torch.exp(c[-1])[:, None, None] + (before[..., None] * Cc).permute(1, 2, 0) @ ys.transpose(0, 1)
    return out
