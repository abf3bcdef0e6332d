"""Plain fp64 implementations of the short convolution, the selective scan and the slot pools, token by
token and slot by slot (torch on the CPU): what the tests compare with."""
from __future__ import annotations

import torch


def f64(x):
    return None if x is None else x.detach().double().cpu()


def spans(B, T, cu):
    """(batch row, first token, one past the last) per sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


# ------------------------------------------------------------------------------- convolution

def conv(x, w, bias=None, h0=None, cu=None, silu=True):
    """(y, final windows); differentiable, fp64."""
    B, T, C = x.shape
    W = w.shape[1]
    runs = spans(B, T, cu)
    h0 = x.new_zeros(len(runs), W - 1, C) if h0 is None else h0
    y, hT = torch.zeros_like(x), []
    rows = []
    for n, (b, lo, hi) in enumerate(runs):
        xp = torch.cat([h0[n], x[b, lo:hi]])
        u = xp.new_zeros(hi - lo, C) if bias is None else bias.expand(hi - lo, C)
        for i in range(W):
            u = u + w[:, i] * xp[i:i + hi - lo]
        rows.append((b, lo, hi, u * torch.sigmoid(u) if silu else u))
        hT.append(xp[hi - lo:])
    y = y.index_put((torch.cat([torch.full((hi - lo,), b) for b, lo, hi, _ in rows]).long(),
                     torch.cat([torch.arange(lo, hi) for _, lo, hi, _ in rows]).long()),
                    torch.cat([u for *_, u in rows]))
    return y, torch.stack(hT)


def conv_grads(x, w, dy, bias=None, h0=None, dhT=None, cu=None, silu=True):
    """(dx, dw, dbias, dh0) by automatic differentiation of `conv`."""
    N = len(spans(x.shape[0], x.shape[1], cu))
    bias = torch.zeros(w.shape[0], dtype=x.dtype) if bias is None else bias
    h0 = x.new_zeros(N, w.shape[1] - 1, x.shape[2]) if h0 is None else h0
    leaves = [t.clone().requires_grad_() for t in (x, w, bias, h0)]
    y, hT = conv(leaves[0], leaves[1], leaves[2], leaves[3], cu, silu)
    loss = (y * dy).sum() + (0 if dhT is None else (hT * dhT).sum())
    return torch.autograd.grad(loss, leaves)


# ------------------------------------------------------------------------------- scan

def heads(x, H):
    """[.., G, d] -> [.., H, d]."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def scan(x, dt, A, B, C, D=None, bias=None, h0=None, cu=None):
    """(y, final states); differentiable, fp64."""
    nb, T, H, dv = x.shape
    runs = spans(nb, T, cu)
    delta = softplus(dt if bias is None else dt + bias)
    Bh, Ch = heads(B, H), heads(C, H)
    h0 = x.new_zeros(len(runs), H, B.shape[-1], dv) if h0 is None else h0
    y, hT, at = [], [], []
    for n, (b, lo, hi) in enumerate(runs):
        S = h0[n]
        for t in range(lo, hi):
            S = S * torch.exp(delta[b, t] * A)[:, None, None] + \
                (delta[b, t][:, None] * Bh[b, t])[:, :, None] * x[b, t][:, None, :]
            y.append((Ch[b, t][:, :, None] * S).sum(1) + (0 if D is None else D[:, None] * x[b, t]))
            at.append((b, t))
        hT.append(S)
    out = torch.zeros_like(x)
    if at:
        out = out.index_put((torch.tensor([b for b, _ in at]), torch.tensor([t for _, t in at])), torch.stack(y))
    return out, torch.stack(hT)


def scan_grads(x, dt, A, B, C, dy, D=None, bias=None, h0=None, dhT=None, cu=None):
    """dict of dx, ddt, dA, dB, dC, dD, dbias, dh0 from the formulas (G_t the gradient of S_t), and of the summed
    magnitudes of what each adds up under "abs"; there also the sums over the tokens of the magnitudes of the
    terms of dA, dbias and dD, as "|dA|" and so on."""
    out = _scan_grads(x, dt, A, B, C, dy, D, bias, h0, dhT, cu)
    a = torch.abs
    sums = {k: out.pop(k) for k in ("|dA|", "|dD|", "|dbias|")}
    mag = _scan_grads(a(x), dt, A, a(B), a(C), a(dy), None if D is None else a(D), bias,
                      None if h0 is None else a(h0), None if dhT is None else a(dhT), cu, magnitude=True)
    out["abs"] = mag
    mag.update(sums)
    return out


def _scan_grads(x, dt, A, B, C, dy, D, bias, h0, dhT, cu, magnitude=False):
    nb, T, H, dv = x.shape
    dk, G_ = B.shape[-1], B.shape[-2]
    runs = spans(nb, T, cu)
    pre = dt if bias is None else dt + bias
    delta, slope = softplus(pre), torch.sigmoid(pre)
    decay = torch.exp(delta * A)
    Aw = A.abs() if magnitude else A
    Bh, Ch = heads(B, H), heads(C, H)
    N = len(runs)
    zero = x.new_zeros(N, H, dk, dv)
    h0, dhT = zero if h0 is None else h0, zero if dhT is None else dhT
    dx, ddt = torch.zeros_like(x), torch.zeros_like(dt)
    dB, dC = (torch.zeros(nb, T, H, dk, dtype=x.dtype) for _ in range(2))
    dA, dD, dbias, aA, aD, ab = (torch.zeros(H, dtype=x.dtype) for _ in range(6))
    dh0 = torch.zeros_like(zero)
    for n, (b, lo, hi) in enumerate(runs):
        states = [h0[n]]
        for t in range(lo, hi):
            states.append(states[-1] * decay[b, t][:, None, None] +
                          (delta[b, t][:, None] * Bh[b, t])[:, :, None] * x[b, t][:, None, :])
        G = dhT[n]
        through = 0.0              # magnitude: what the sum over a segment of tokens that dg comes from adds up
        for t in reversed(range(lo, hi)):
            G = G + Ch[b, t][:, :, None] * dy[b, t][:, None, :]
            S = states[t - lo + 1]
            dC[b, t] = (S * dy[b, t][:, None, :]).sum(-1)
            dB[b, t] = delta[b, t][:, None] * (G * x[b, t][:, None, :]).sum(-1)
            u = (G * Bh[b, t][:, :, None]).sum(1)
            dx[b, t] = delta[b, t][:, None] * u + (0 if D is None else D[:, None] * dy[b, t])
            dg = decay[b, t] * (G * states[t - lo]).sum((-1, -2))
            xu = (x[b, t] * u).sum(-1)
            if magnitude:
                through = through + (Ch[b, t] * dC[b, t]).sum(-1) + delta[b, t] * xu
                dg = dg + through
            ddt[b, t] = (xu + Aw * dg) * slope[b, t]
            dA += delta[b, t] * dg
            dbias += ddt[b, t]
            dD += (x[b, t] * dy[b, t]).sum(-1)
            aA += (delta[b, t] * dg).abs()
            ab += ddt[b, t].abs()
            aD += (x[b, t] * dy[b, t]).abs().sum(-1)
            G = decay[b, t][:, None, None] * G
        dh0[n] = G
    def group(g):
        return g.unflatten(2, (G_, H // G_)).sum(3)
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": group(dB), "dC": group(dC), "dD": dD, "dbias": dbias, "dh0": dh0,
            "|dA|": aA, "|dD|": aD, "|dbias|": ab}


# ------------------------------------------------------------------------------- slots

def compact(refs, table):
    """(refs, table, used, [(from, to)]) after moving the used slots together; host lists."""
    refs = list(refs)
    used = sum(r > 0 for r in refs)
    low = [s for s in range(used) if refs[s] <= 0]
    high = [s for s in range(used, len(refs)) if refs[s] > 0]
    where = {s: s for s in range(len(refs)) if refs[s] > 0}
    moves = list(zip(high, low))
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
        where[a] = b
    return refs, [where.get(s, -1) for s in table], used, moves


def fork(refs, parents):
    """(refs, children, sources): sources None: zeros; host lists."""
    before, refs = list(refs), list(refs)
    free = [s for s, r in enumerate(refs) if r <= 0]
    children, sources = [], []
    for i, p in enumerate(parents):
        children.append(free[i] if i < len(free) else -1)
        sources.append(p if 0 <= p < len(before) and before[p] > 0 else None)
        if children[-1] >= 0:
            refs[children[-1]] = 1
    return refs, children, sources
