"""Plain fp64 implementations of linear attention with one decay per head and of the 8-bit state
cache, token by token and element by element (numpy, CPU): what the tests compare with."""
from __future__ import annotations

import numpy as np
import torch


def np64(x):
    return None if x is None else x.detach().double().cpu().numpy()


def spans(B, T, cu):
    """(batch row, first token, one past the last) per sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, g, h0=None, cu=None, scale=1.0):
    """(o, final states) of numpy fp64 inputs [B, T, H, d], g [H]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    runs = spans(B, T, cu)
    lam = np.exp(g)[:, None, None]
    o = np.zeros((B, T, H, dv))
    hT = np.zeros((len(runs), H, dk, dv)) if h0 is None else h0.copy()
    for n, (b, lo, hi) in enumerate(runs):
        S = hT[n]
        for t in range(lo, hi):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = scale * np.einsum("hc,hcd->hd", q[b, t], S)
        hT[n] = S
    return o, hT


def backward(q, k, v, g, do, h0=None, dhT=None, cu=None, scale=1.0):
    """(dq, dk, dv, gradient of the initial states)."""
    B, T, H, dk_ = q.shape
    dv_ = v.shape[-1]
    runs = spans(B, T, cu)
    lam = np.exp(g)[:, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dh0 = np.zeros((len(runs), H, dk_, dv_)) if dhT is None else dhT.copy()
    for n, (b, lo, hi) in enumerate(runs):
        S = np.zeros((H, dk_, dv_)) if h0 is None else h0[n]
        for t in range(lo, hi):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            dq[b, t] = scale * np.einsum("hcd,hd->hc", S, do[b, t])
        G = dh0[n]                                   # gradient of the state after token t
        for t in range(hi - 1, lo - 1, -1):
            G = G + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dk[b, t] = np.einsum("hcd,hd->hc", G, v[b, t])
            dv[b, t] = np.einsum("hcd,hc->hd", G, k[b, t])
            G = lam * G
        dh0[n] = G
    return dq, dk, dv, dh0


def forward_abs(q, k, v, g, h0=None, cu=None, scale=1.0):
    """The sums of the magnitudes of everything `forward` adds up: what rounding errors scale with."""
    a = np.abs
    return forward(a(q), a(k), a(v), g, None if h0 is None else a(h0), cu, abs(scale))


def backward_abs(q, k, v, g, do, h0=None, dhT=None, cu=None, scale=1.0):
    a = np.abs
    return backward(a(q), a(k), a(v), g, a(do), None if h0 is None else a(h0),
                    None if dhT is None else a(dhT), cu, abs(scale))


# ------------------------------------------------------------------------------- state cache

MOST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def e4m3_values():
    """The value of each byte as an e4m3 number (1 sign, 4 exponent, 3 mantissa bits, bias 7)."""
    out = np.zeros(256)
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[i] = np.nan if e == 15 and m == 7 else (-x if i & 128 else x)
    return out


def quantise(x, group, dtype):
    """(values of the codes, fp32 scales) of fp32 states x [..., dv]: scale = max|x| times the fp32
    reciprocal of the largest code; nearest code, ties to even."""
    x = np.asarray(x, dtype=np.float32)
    most = MOST[dtype]
    y = x.reshape(x.shape[:-1] + (-1, group))
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(y).max(-1)
        bad = ~np.isfinite(y).all(-1)
        scale = np.where(bad, np.float32(np.nan), (amax * (np.float32(1) / np.float32(most))).astype(np.float32))
        div = np.where(np.isfinite(scale) & (scale > 0), scale, 1.0).astype(np.float64)[..., None]
        r = np.where((bad | (scale == 0))[..., None], 0.0, y.astype(np.float64)) / div
    if dtype == torch.int8:
        c = np.rint(r)
    else:
        size = np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -6)))
        ulp = 2.0 ** (size - 3)
        c = np.rint(r / ulp) * ulp
    return np.clip(c, -most, most).reshape(x.shape), scale.astype(np.float32)


def code_values(codes: torch.Tensor):
    """What a code tensor's bytes stand for, in fp64."""
    raw = codes.detach().cpu().view(torch.uint8).numpy()
    if codes.dtype == torch.int8:
        return raw.view(np.int8).astype(np.float64)
    return e4m3_values()[raw]
