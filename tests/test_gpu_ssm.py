"""The selective scan on the GPU against the fp64 reference: prefill and gradients over types, head sizes,
groups, lengths (empty and single-token sequences, chunk borders, several segments), states and strides.

Tolerances.  bf16 inputs enter the products exactly; states and weighted scores are read as two bf16 terms, each
rounded to nearest, so a term is off by at most 2^-17 of itself; a result adds the state's part (one such
reading) and the scores' part (one), and fp32 accumulation over fewer than 2^9 terms adds less than 2^-15 of the
summed magnitudes in the worst case.  So |error| <= 2^-14 of the summed magnitudes, and for fp32 inputs, whose
products are fp32 throughout, 2^-15 (accumulation, and decays of relative error 2^-23 |log decay|, whose
contributions are then small).  An output in bf16 adds its rounding, at most 2^-8 of the value.  The errors are
also small on average: their root mean square is held below 2^-14 (fp32: 2^-17) of the values' and the
rounding's."""
import pytest
import torch

import ssm_ref as R
from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV, say

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def make(dtype, lens, H, G, dk, dv, packed, state, skip=True, bias=True, seed=0, scale_dt=1.0, wide=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    N = len(lens)
    B, T = (1, sum(lens)) if packed else (N, lens[0])
    pad = 16 if wide else 0
    row = r(B, T, H * dv + 2 * G * dk + pad).to(dtype)
    cuts = [0]
    for n in lens:
        cuts.append(cuts[-1] + n)
    d = dict(row=row, dt=(scale_dt * r(B, T, H)).to(dtype), A=-(0.5 + 8 * torch.rand(H, generator=g)), D=r(H) if skip else None,
             bias=-2 + r(H) if bias else None, h0=r(N, H, dk, dv) if state else None,
             cu=torch.tensor(cuts, dtype=torch.int32) if packed else None, dy=r(B, T, H, dv).to(dtype),
             dhT=r(N, H, dk, dv) if state else None)
    x = row[..., :H * dv].unflatten(-1, (H, dv))
    Bm = row[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk))
    Cm = row[..., H * dv + G * dk:H * dv + 2 * G * dk].unflatten(-1, (G, dk))
    d["ref"] = dict(x=R.f64(x), dt=R.f64(d["dt"]), A=R.f64(d["A"]), B=R.f64(Bm), C=R.f64(Cm), D=R.f64(d["D"]),
                    bias=R.f64(d["bias"]), h0=R.f64(d["h0"]), cu=None if d["cu"] is None else d["cu"].tolist())
    dev = d["row"].to(DEV)
    d["x"] = dev[..., :H * dv].unflatten(-1, (H, dv))
    d["B"] = dev[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk))
    d["C"] = dev[..., H * dv + G * dk:H * dv + 2 * G * dk].unflatten(-1, (G, dk))
    for k in ("dt", "A", "D", "bias", "h0", "cu", "dy", "dhT"):
        d[k] = None if d[k] is None else d[k].to(DEV)
    return d


def check(name, got, ref, mag, in_dtype):
    out = torch.finfo(got.dtype).eps / 2
    k, rms_k = (2.0 ** -14, 2.0 ** -14) if in_dtype == bf else (2.0 ** -15, 2.0 ** -17)
    got, ref = got.double().cpu(), ref
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    if not ref.numel():
        return
    err = (got - ref).abs()
    worst = (err - out * ref.abs() - k * mag).max().item()
    rms, size = err.pow(2).mean().sqrt().item(), ref.pow(2).mean().sqrt().item()
    say(f"  {name}: rms {rms / max(size, 1e-300):.2e}, worst beyond {worst:.2e}")
    assert worst <= 0, (name, worst)
    assert rms <= (out + rms_k) * size + 1e-30, (name, rms, size)


def check_sum(name, got, ref, terms):
    """dA, dD, dbias: sums over the tokens of terms of either sign.  A sum may be far smaller than its terms, so its
    error is held against their summed magnitudes and not against itself: 2^-16 of them (a term's products are exact
    or two bf16 terms, 2^-17; fp32 sums over up to 512 tokens, 2^-18 on average; the sums over segments are fp64)."""
    worst = ((got.double().cpu() - ref).abs() / terms.clamp(min=1e-300)).max().item()
    say(f"  {name}: {worst:.2e} of its terms")
    assert worst <= 2.0 ** -16, (name, worst)


def forward(d, **kw):
    return K.kda_ssm_chunk_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"],
                               initial_state=d["h0"], cu_seqlens=d["cu"], **kw)


def backward(d, **kw):
    return K.kda_ssm_chunk_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], D=d["D"], dt_bias=d["bias"],
                               initial_state=d["h0"], d_final_state=d["dhT"], cu_seqlens=d["cu"], **kw)


def check_forward(d, dtype, **kw):
    y, hT = forward(d, **kw)
    torch.cuda.synchronize()
    y_ref, h_ref = R.scan(**d["ref"])
    mag = {k: (v.abs() if isinstance(v, torch.Tensor) and k not in ("dt", "A", "bias") else v) for k, v in d["ref"].items()}
    y_mag, h_mag = R.scan(**mag)
    check("y", y, y_ref, y_mag, dtype)
    check("state", hT, h_ref, h_mag, f32)       # three terms: fp32 accuracy whatever the inputs
    return y, hT


def check_backward(d, dtype, **kw):
    got = backward(d, **kw)
    torch.cuda.synchronize()
    ref = R.scan_grads(dy=R.f64(d["dy"]), dhT=R.f64(d["dhT"]), **d["ref"])
    for name, t in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dbias", "dh0"), got):
        if t is not None and name in ("dA", "dD", "dbias"):
            check_sum(name, t, ref[name], ref["abs"][f"|{name}|"])
        elif t is not None:
            check(name, t, ref[name], ref["abs"][name], dtype)
    assert (got[5] is None) == (d["D"] is None) and (got[6] is None) == (d["bias"] is None)
    assert (got[7] is None) == (d["h0"] is None)
    return got


SIZES = [(64, 64), (128, 64), (64, 128), (128, 128)]
BATCHES = [
    (dict(lens=[1], packed=False, state=True), (2, 1)),
    (dict(lens=[63, 63], packed=False, state=False), (3, 1)),
    (dict(lens=[64], packed=False, state=True), (2, 2)),
    (dict(lens=[65], packed=False, state=True), (4, 2)),
    (dict(lens=[5, 0, 1, 130, 64, 0, 37], packed=True, state=True), (6, 2)),
    (dict(lens=[200, 70], packed=True, state=False), (5, 1)),
]


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("batch,hg", BATCHES)
def test_forward(dtype, dk, dv, batch, hg):
    d = make(dtype, H=hg[0], G=hg[1], dk=dk, dv=dv, **batch)
    check_forward(d, dtype)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("batch,hg", BATCHES)
def test_backward(dtype, dk, dv, batch, hg):
    d = make(dtype, H=hg[0], G=hg[1], dk=dk, dv=dv, **batch)
    check_backward(d, dtype)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("lens,packed", [([1290], False), ([1100, 0, 1, 513, 64], True), ([512, 1024, 600], True)])
def test_segments(dtype, lens, packed):
    """Sequences that run in several segments, forward and backward."""
    d = make(dtype, lens, H=3, G=1, dk=64, dv=64, packed=packed, state=True, scale_dt=2.0)
    check_forward(d, dtype)
    check_backward(d, dtype)


@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_output_types_and_options(dtype, y_dtype):
    d = make(dtype, [77, 77], H=4, G=2, dk=64, dv=64, packed=False, state=False, skip=False, bias=False)
    y, _ = check_forward(d, dtype, y_dtype=y_dtype)
    assert y.dtype == y_dtype
    check_backward(d, dtype)


def test_extreme_decays():
    """Steps from nothing (delta 2^-60) to a full reset (log-decay -1e5) side by side: decays between close
    tokens must not suffer from strong ones before them, and no sum may overflow."""
    for dtype in (bf, f32):
        d = make(dtype, [300], H=4, G=2, dk=64, dv=64, packed=False, state=True, bias=False)
        dt = torch.where(torch.rand(d["dt"].shape, generator=torch.Generator().manual_seed(5)) < 0.03, 1e4, -1.0)
        dt[:, ::7] = -40.0
        d["dt"] = dt.to(dtype).to(DEV)
        d["ref"]["dt"] = R.f64(d["dt"])
        # delta up to 1e4 and |A| up to 8.5: |log decay| up to 8.5e4
        check_forward(d, dtype)
        check_backward(d, dtype)


def test_gradients_into_one_row_buffer():
    """dx, dB and dC written side by side, as the convolution's gradients read them; what lies between stays."""
    H, G, dk, dv = 4, 2, 64, 64
    d = make(bf, [130, 70], H, G, dk, dv, packed=True, state=True)
    want = backward(d)
    row = torch.full((1, 200, H * dv + 2 * G * dk + 16), 7.0, dtype=bf, device=DEV)
    dx, dB = row[..., :H * dv].unflatten(-1, (H, dv)), row[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk))
    dC = row[..., H * dv + G * dk:H * dv + 2 * G * dk].unflatten(-1, (G, dk))
    got = backward(d, dx=dx, dB=dB, dC=dC)
    torch.cuda.synchronize()
    assert got[0] is dx and got[3] is dB and got[4] is dC
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert (row[..., -16:] == 7.0).all()


def test_rows_behind_the_last_sequence():
    """A packed buffer with more rows than the sequences hold: they are neither read into results nor written."""
    d = make(bf, [70, 9, 100], H=4, G=2, dk=64, dv=64, packed=True, state=True)
    want_y, want_h = forward(d)
    want = backward(d)
    cut = 79
    d["cu"] = d["cu"][:3].contiguous()
    d["h0"], d["dhT"] = d["h0"][:2].contiguous(), d["dhT"][:2].contiguous()
    y = torch.full_like(want_y, 3.0)
    y, hT = forward(d, y=y)
    outs = {k: torch.full_like(t.contiguous(), 3.0) for k, t in (("dx", d["x"]), ("ddt", d["dt"]), ("dB", d["B"]), ("dC", d["C"]))}
    got = backward(d, **outs)
    torch.cuda.synchronize()
    assert torch.equal(y[:, :cut], want_y[:, :cut]) and torch.equal(hT, want_h[:2]) and (y[:, cut:] == 3.0).all()
    for i, k in ((0, "dx"), (1, "ddt"), (3, "dB"), (4, "dC")):
        assert torch.equal(got[i][:, :cut], want[i][:, :cut]), k
        assert (got[i][:, cut:] == 3.0).all(), k


def test_no_tokens():
    for packed in (False, True):
        d = make(f32, [0, 0], H=2, G=1, dk=64, dv=64, packed=packed, state=True, wide=False)
        y, hT = forward(d)
        got = backward(d)
        torch.cuda.synchronize()
        assert torch.equal(hT, d["h0"]) and torch.equal(got[7], d["dhT"]) and y.numel() == 0
        for i in (2, 5, 6):
            assert (got[i] == 0).all()


def test_in_place_final_state_and_repeats():
    """The final state in the initial state's buffer, with and without segments; equal bits call after call."""
    for lens in ([100], [1500]):
        d = make(bf, lens, H=3, G=1, dk=128, dv=64, packed=False, state=True)
        y, hT = forward(d)
        h = d["h0"].clone()
        d2 = dict(d, h0=h)
        y2, h2 = forward(d2, final_state=h)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(hT, h2) and h2 is h
        a, b = backward(d), backward(d)
        torch.cuda.synchronize()
        for s, t in zip(a, b):
            assert torch.equal(s, t)
