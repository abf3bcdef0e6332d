"""CPU pins of the fp64 references in linear_ref.py: gradients against central differences (the
outputs are linear in each input, so these are exact up to fp64 rounding), closed forms, and the
e4m3 table against torch's."""
import numpy as np
import pytest
import torch

import linear_ref as R


def case(seed, B=2, T=7, H=2, dk=3, dv=4, cu=None):
    r = np.random.default_rng(seed)
    N = B if cu is None else len(cu) - 1
    d = dict(q=r.standard_normal((B, T, H, dk)), k=r.standard_normal((B, T, H, dk)),
             v=r.standard_normal((B, T, H, dv)), h0=r.standard_normal((N, H, dk, dv)))
    return d, -np.exp(r.standard_normal(H)), r.standard_normal((B, T, H, dv)), \
        r.standard_normal((N, H, dk, dv))


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_gradients_against_differences(cu):
    d, g, do, dhT = case(1, B=1 if cu else 2, cu=cu)
    scale = 0.7
    grads = dict(zip(("q", "k", "v", "h0"),
                     R.backward(d["q"], d["k"], d["v"], g, do, d["h0"], dhT, cu, scale)))

    def loss(**over):
        x = {**d, **over}
        o, hT = R.forward(x["q"], x["k"], x["v"], g, x["h0"], cu, scale)
        return (o * do).sum() + (hT * dhT).sum()

    r = np.random.default_rng(2)
    for name in ("q", "k", "v", "h0"):
        e = r.standard_normal(d[name].shape)
        diff = (loss(**{name: d[name] + e}) - loss(**{name: d[name] - e})) / 2
        assert abs(diff - (grads[name] * e).sum()) <= 1e-10 * max(1.0, abs(diff)), name


def test_closed_forms():
    d, g, _, _ = case(3)
    # no decay: plain prefix sums of k v^T
    o, hT = R.forward(d["q"], d["k"], d["v"], np.zeros(2))
    S = np.cumsum(np.einsum("bthc,bthd->bthcd", d["k"], d["v"]), axis=1)
    assert np.allclose(o, np.einsum("bthc,bthcd->bthd", d["q"], S)) and np.allclose(hT, S[:, -1])
    # full decay: each token sees itself alone
    o, hT = R.forward(d["q"], d["k"], d["v"], np.full(2, -np.inf), d["h0"])
    assert np.allclose(o, (d["q"] * d["k"]).sum(-1, keepdims=True) * d["v"])
    # no tokens: the state passes through
    _, hT = R.forward(d["q"][:, :0], d["k"][:, :0], d["v"][:, :0], g, d["h0"])
    assert np.array_equal(hT, d["h0"])


def test_e4m3_table_and_rounding():
    t = R.e4m3_values()
    ref = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref, equal_nan=True)
    finite = np.sort(np.unique(t[np.isfinite(t)]))
    x = np.random.default_rng(0).standard_normal(4096).astype(np.float32)
    c, s = R.quantise(x.reshape(32, 128), 128, torch.float8_e4m3fn)
    assert np.isin(c, finite).all()
    r = x.reshape(32, 128).astype(np.float64) / s.astype(np.float64)
    best = np.abs(r[..., None] - finite).min(-1)
    assert np.all(np.abs(c - r) <= best * (1 + 1e-12))
