"""How far an infinity or a NaN in one token of a selective scan or a convolution reaches: what the formulas give it, and
beside that 63 tokens of its own sequence on either side at most (the convolution: none); never another sequence, whose
results keep their bits.  What stands in rows of no sequence reaches nothing, and a dt of minus infinity is a token that
leaves the state alone."""
import pytest
import torch

import ssm_ref as R
from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV
from test_gpu_ssm import backward, bf, check_backward, check_forward, f32, forward, make

pytestmark = pytest.mark.gpu
LENS, AT = [70, 1300, 0, 65], 1010                   # the token lies in the second sequence
LO, HI = LENS[0], LENS[0] + LENS[1]
OTHERS = torch.tensor([0, 2, 3])
nan, inf = float("nan"), float("inf")
# Outputs that the formulas let an input of token AT reach: the tokens from it on, up to it, all, or itself alone; and
# whether it gets to the final state (hT) and to the initial state's gradient (dh0).
REACH = dict(x=dict(y="from", dC="from", dB="self", ddt="from", hT="yes"),
             B=dict(y="from", dC="from", dx="self", ddt="from", hT="yes"),
             C=dict(y="self", dx="to", dB="to", ddt="to", dh0="yes"),
             dy=dict(dx="to", dB="to", dC="self", ddt="to", dh0="yes"),
             dt=dict(y="from", dC="from", dx="all", dB="all", ddt="all", hT="yes", dh0="yes"))
# e^(delta A) of an infinite delta is 0: what lies before such a token is cut off from what lies behind it
RESET = dict(y="from", dC="from", dx="self", dB="self", ddt="from", hT="yes")


def may_reach(how, near):
    t = torch.arange(sum(LENS))
    inside = (t >= LO) & (t < HI)
    formula = {"none": t < 0, "self": t == AT, "from": t >= AT, "to": t <= AT, "all": t >= 0}[how]
    return inside & (formula | ((t - AT).abs() <= near))


def results(d):
    y, hT = forward(d)
    dx, ddt, _, dB, dC, _, _, dh0 = backward(d)
    torch.cuda.synchronize()
    return dict(y=y, dx=dx, ddt=ddt, dB=dB, dC=dC), hT, dh0


def compare(clean, dirty, reach, near=63):
    for (k, t), c in zip(dirty[0].items(), clean[0].values()):
        t, c = t[0].flatten(1).cpu(), c[0].flatten(1).cpu()
        may = may_reach(reach.get(k, "none"), near)
        assert bool((torch.isfinite(t).all(1) | may).all()), (k, (~torch.isfinite(t).all(1) & ~may).nonzero().flatten().tolist())
        other = (torch.arange(sum(LENS)) < LO) | (torch.arange(sum(LENS)) >= HI)
        assert torch.equal(t[other], c[other]), k


@pytest.mark.parametrize("name,bad", [(name, bad) for name in ("x", "B", "C", "dy") for bad in (nan, inf, -inf)] + [("dt", nan), ("dt", inf)])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("H,dk,dv", [(2, 64, 128), (2, 128, 64), (130, 64, 64)])           # in segments; whole
def test_reach(H, dk, dv, dtype, name, bad):
    d = make(dtype, LENS, H, 1, dk, dv, packed=True, state=True, seed=70)
    clean = results(d)
    if name == "dt":
        d["dt"][0, AT] = bad
    else:
        d[name][0, AT, :, 5] = bad
    dirty = results(d)
    reach = RESET if name == "dt" and bad == inf else REACH[name]
    compare(clean, dirty, reach)
    for i, k in ((1, "hT"), (2, "dh0")):
        assert torch.equal(dirty[i][OTHERS], clean[i][OTHERS]), k
        if k not in reach:
            assert bool(torch.isfinite(dirty[i]).all()), k


@pytest.mark.parametrize("value", [-inf, -3e38])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_steps_of_nothing(dk, dv, dtype, value):
    """dt of minus infinity, or of the type's lowest values: delta is 0, the token neither writes nor decays."""
    d = make(dtype, [200, 40], 4, 2, dk, dv, packed=True, state=True, seed=71)
    for sel in (slice(0, 3), slice(60, 70), slice(190, 240, 3)):
        d["dt"][0, sel] = value
    d["ref"]["dt"] = R.f64(d["dt"])
    check_forward(d, dtype)
    got = check_backward(d, dtype)
    assert bool((got[1][0, 60:70] == 0).all())
    # and one token at a time
    state = d["h0"][:1].clone()
    x, dt, B, C = (d[k][:, 60].contiguous() for k in ("x", "dt", "B", "C"))
    K.kda_ssm_decode_step(x, dt, d["A"], B, C, state, dt_bias=d["bias"])
    torch.cuda.synchronize()
    assert torch.equal(state, d["h0"][:1])


@pytest.mark.parametrize("bad", [nan, inf])
@pytest.mark.parametrize("dtype", [bf, f32])
def test_rows_of_no_sequence(dtype, bad):
    """A padded buffer whose last rows hold anything."""
    d = make(dtype, [70, 1100, 60], 4, 2, 64, 64, packed=True, state=True, seed=72)
    d["cu"], d["h0"], d["dhT"] = d["cu"][:3].contiguous(), d["h0"][:2].contiguous(), d["dhT"][:2].contiguous()
    kept = lambda: [t[:, :1170] if t.dim() > 2 and t.shape[1] == 1230 else t for t in (*forward(d), *backward(d))]   # noqa: E731
    clean = kept()
    row = d["x"]._base
    for t in (row, d["dt"], d["dy"]):
        t[:, 1170:] = bad
    dirty = kept()
    w = torch.randn(64, 4, generator=torch.Generator().manual_seed(1)).to(DEV)
    x, dy = row[..., :64], d["dy"].flatten(2)[..., :64]
    whole = [*K.kda_conv_fwd(x, w, cu_seqlens=d["cu"], output_final_state=True), *K.kda_conv_bwd(x, w, dy, cu_seqlens=d["cu"])[:2]]
    short = [t[:, :1170].contiguous() for t in (x, dy)]
    want = [*K.kda_conv_fwd(short[0], w, cu_seqlens=d["cu"], output_final_state=True), *K.kda_conv_bwd(short[0], w, short[1], cu_seqlens=d["cu"])[:2]]
    torch.cuda.synchronize()
    for a, b in zip(clean + want, dirty + whole):
        assert torch.equal(a, b[:, :1170] if b.dim() == 3 and b.shape[1] == 1230 else b)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("bad", [nan, inf, -inf])
@pytest.mark.parametrize("name", ["x", "dy"])
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("C", [64, 67])
def test_convolution(C, dtype, name, bad, silu):
    """The formulas' reach and no more: W - 1 tokens either way, of the one channel."""
    g = torch.Generator().manual_seed(73)
    W, T = 4, sum(LENS)
    d = dict(x=torch.randn(1, T, C, generator=g).to(dtype).to(DEV), dy=torch.randn(1, T, C, generator=g).to(dtype).to(DEV))
    w, b = torch.randn(C, W, generator=g).to(DEV), torch.randn(C, generator=g).to(DEV)
    cu = torch.tensor([0, 70, 1370, 1370, 1435], dtype=torch.int32, device=DEV)

    def run():
        y, hT = K.kda_conv_fwd(d["x"], w, b, cu_seqlens=cu, silu=silu, output_final_state=True)
        dx, dw, db, _ = K.kda_conv_bwd(d["x"], w, d["dy"], b, cu_seqlens=cu, silu=silu)
        torch.cuda.synchronize()
        return dict(y=y, dx=dx), hT, dw, db

    clean = run()
    at = AT - AT % 16                                # the first token of a walk: its neighbours belong to another
    d[name][0, at, 9] = bad
    dirty = run()
    t = torch.arange(T, device=DEV)
    reach = {("x", "y"): (t >= at) & (t < at + W), ("x", "dx"): ((t - at).abs() < W) & silu, ("dy", "dx"): (t <= at) & (t > at - W)}
    for k, got in dirty[0].items():
        same = (got == clean[0][k])[0]
        may = reach.get((name, k), t < 0)
        assert bool(same[:, torch.arange(C, device=DEV) != 9].all()) and bool((same[:, 9] | may).all()), k
    assert torch.equal(dirty[1], clean[1])
    for i in (2, 3):
        other = torch.arange(C, device=DEV) != 9
        assert torch.equal(dirty[i][other], clean[i][other])
