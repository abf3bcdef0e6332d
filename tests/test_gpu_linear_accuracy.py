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


def relative(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def exact_states(k, v, g, h0):
    """Final states of [B, T, H, d] inputs, token by token in fp64 on the GPU."""
    lam = torch.exp(g.double())[:, None, None]
    S = h0.double()
    for t in range(k.shape[1]):
        S = lam * S + k[:, t].double()[..., None] * v[:, t].double()[..., None, :]
    return S


@pytest.mark.parametrize("B,H", [(64, 4), (1, 3)])      # whole sequences, and segments
def test_states_hold_fp32_accuracy(B, H):
    """bf16 inputs, slow decays: each of the 192 additions to a state (2048 tokens in steps of 32, three terms
    each) rounds it by 2^-24 * 1.5 / sqrt(12) of itself (rms), on the way to a state that grows like the root
    of the tokens: 2^-24 * 0.43 * sqrt(192 / 2) = 2.5e-7 in all; four times that.  Two terms instead of three
    would leave out 2^-17 of each addend and more, 2.6e-6."""
    T = 2048
    gen = torch.Generator("cpu").manual_seed(7)
    q, k, v, do = (torch.randn((B, T, H, 64), generator=gen).to(BF).to(DEV) for _ in range(4))
    g = torch.tensor([-1e-4, -1e-3, -1e-2, -1e-4][:H], device=DEV)
    h0, dhT = (torch.randn((B, H, 64, 64), generator=gen).to(DEV) for _ in range(2))
    tol = 4 * 2.0 ** -24 * 0.43 * 96 ** 0.5
    _, S = K.kda_linear_chunk_fwd(q, k, v, g, initial_state=h0)
    err = relative(S, exact_states(k, v, g, h0))
    say(f"  final state {err:.2e} of {tol:.2e}")
    assert err <= tol
    dh0 = K.kda_linear_chunk_bwd(q, k, v, g, do, initial_state=h0, d_final_state=dhT)[3]
    # G_t adds q_t do_t^T before its decay: the recurrence run from the back, decayed once more at the end
    lam = torch.exp(g.double())[:, None, None]
    ref = dhT.double()
    for t in range(T - 1, -1, -1):
        ref = lam * (ref + q[:, t].double()[..., None] * do[:, t].double()[..., None, :])
    err = relative(dh0, ref)
    say(f"  d_initial_state {err:.2e} of {tol:.2e}")
    assert err <= tol
