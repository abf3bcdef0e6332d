"""How far an infinity or a NaN in one token of a linear-attention prefill reaches: what the formulas give it,
and on their masked side 64 tokens of its own sequence at most (before it for o and dq, after it for dk and dv)."""
import pytest
import torch

from gated_delta_rule_60_amd import kda as K
from test_gpu_linear import BF, F32, dev, make

pytestmark = pytest.mark.gpu
LENS, AT = [70, 1300, 0, 65], 1010                   # the token lies in the second sequence
LO, HI = LENS[0], LENS[0] + LENS[1]
# outputs that the formulas let an input of token AT reach: the tokens from it on, up to it, or itself alone
REACH = dict(q=dict(o="self", dk="to", dv="to"), k=dict(o="from", dq="from", dv="self"),
             v=dict(o="from", dq="from", dk="self"), do=dict(dq="self", dk="to", dv="to"))


def may_reach(how):
    t = torch.arange(sum(LENS))
    inside = (t >= LO) & (t < HI)
    return {"none": t < 0, "self": t == AT, "from": inside & (t >= AT - 64), "to": inside & (t <= AT + 64)}[how]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [2, 80])                # in segments; whole
def test_reach(H, dtype, name, bad):
    d = make(1, 0, H, 64, 128, dtype, lens=LENS, seed=70)
    d["g"] = torch.linspace(-0.2, 0.0, H)
    d[name][0, AT, :, 5] = bad
    x = {n: dev(t) for n, t in d.items()}
    o, S = K.kda_linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], cu_seqlens=x["cu"])
    dq, dk, dv, dh = K.kda_linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], initial_state=x["h0"],
                                            d_final_state=x["dhT"], cu_seqlens=x["cu"])
    torch.cuda.synchronize()
    for out, t in dict(o=o, dq=dq, dk=dk, dv=dv).items():
        finite = torch.isfinite(t)[0].flatten(1).all(1).cpu()
        may = may_reach(REACH[name].get(out, "none"))
        assert bool((finite | may).all()), (out, (~finite & ~may).nonzero().flatten().tolist())
    seqs = torch.tensor([0, 2, 3])
    assert bool(torch.isfinite(S[seqs]).all()) and bool(torch.isfinite(dh[seqs]).all())
    if name in ("q", "do"):
        assert bool(torch.isfinite(S).all())
    else:
        assert bool(torch.isfinite(dh).all())
