"""What linear attention's states hold over many calls and many tokens: a decay applied thousands of times
must not carry its own rounding along, and final states keep fp32 accuracy."""
import numpy as np
import pytest
import torch

from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CALLS = 10000


def worst_rounding(g0, T):
    """The fp32 log-decay near g0 whose factor over T tokens has the largest relative rounding in fp32."""
    g = (g0 * (1 + 1e-3 * np.arange(200))).astype(np.float32)
    lam = np.exp(T * g.astype(np.float64))
    return float(g[np.argmax(np.abs(lam.astype(np.float32) / lam - 1))])


def decays(T):
    return np.array([worst_rounding(g0 / T, T) for g0 in (-1e-3, -1e-4, -1e-5)])


def check_decayed(S, h0, g, T, roundings, form):
    """S against e^(CALLS T g) h0, by norms over a head's state.  Each call rounds a state element
    `roundings` times, off by 2^-23 / sqrt(12) of it (rms) as long as the roundings are independent:
    2^-23 sqrt(roundings CALLS / 12) in all.  For slow decays they are not: a call takes D = e 2^23 to
    e 2^24 steps of the last place off an element (e = T |g|), D changes by e D per call, so its fraction
    (the rounding) runs through one step in 1 / (e D) calls; the incomplete run leaves at most an eighth of
    that many steps: 2^-46 / (8 e^2).  Four times their sum; a decay held in fp32 alone is off by up to
    2^-25 in every call, 3e-4 in all."""
    S, h0 = S.double().cpu().numpy(), h0.double().cpu().numpy()
    for h, gh in enumerate(g):
        e = T * abs(gh)
        ref = np.exp(CALLS * T * gh) * h0[:, h]
        err = np.linalg.norm(S[:, h] - ref) / np.linalg.norm(ref)
        tol = 4 * (2.0 ** -23 * np.sqrt(roundings * CALLS / 12) + 2.0 ** -46 / (8 * e * e))
        say(f"  {form}, e = {e:.1e}: {err:.2e} of {tol:.2e}")
        assert err <= tol, (form, gh)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_decay_over_many_steps(dtype):
    g = decays(1)
    z = torch.zeros((2, 3, 64), dtype=dtype, device=DEV)
    gen = torch.Generator("cpu").manual_seed(1)
    h0 = torch.randn((2, 3, 64, 64), generator=gen).to(DEV)
    S, gd = h0.clone(), torch.tensor(g, dtype=F32, device=DEV)
    o = torch.empty_like(z)
    for _ in range(CALLS):
        K.kda_linear_decode_step(z, z, z, gd, S, o=o)
    torch.cuda.synchronize()
    check_decayed(S, h0, g, 1, 1, "decode")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 17, 64, 65])
def test_prefill_decay_over_many_calls(T, dtype):
    """A prompt fed in short pieces, each from the state the one before left: a partial chunk's decay and
    the one pending at the end round the state twice."""
    g = decays(T)
    z = torch.zeros((2, T, 3, 64), dtype=dtype, device=DEV)
    gen = torch.Generator("cpu").manual_seed(2)
    h0 = torch.randn((2, 3, 64, 64), generator=gen).to(DEV)
    S, gd = h0.clone(), torch.tensor(g, dtype=F32, device=DEV)
    o = torch.empty_like(z)
    for _ in range(CALLS):
        K.kda_linear_chunk_fwd(z, z, z, gd, initial_state=S, final_state=S, o=o)
    torch.cuda.synchronize()
    check_decayed(S, h0, g, T, 2, f"prefill of {T}")
