"""The selective scan's workspace size never falls as tokens or sequences grow: what serves the largest batch of a
model serves every smaller one (CPU)."""
import random

import pytest
import torch

from gated_delta_rule_60_amd import kda as K

bf, f32 = torch.bfloat16, torch.float32
HEADS = [(32, 1, 128, 64), (32, 1, 128, 128), (8, 8, 128, 128), (4, 2, 64, 64), (1, 1, 64, 64), (6, 2, 64, 128),
         (24, 8, 128, 64), (80, 1, 64, 64), (300, 1, 64, 64), (300, 300, 64, 128)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("backward", [False, True])
def test_never_falls(heads, dtype, backward):
    size = lambda n, t: K.kda_ssm_chunk_workspace_size(n, t, *heads, dtype, backward)   # noqa: E731
    r = random.Random(f"{heads}{dtype}{backward}")
    pick = lambda top: int(top ** r.random())                                           # noqa: E731
    for n in (1, 2, 3, 15, 16, pick(300), pick(300)):                # along the tokens, close together and far apart
        last = 0
        for t in sorted([*range(0, 20000, 41), *(pick(200000) for _ in range(300)), 16320, 16384, 65536]):
            need = size(n, t)
            assert need >= last, (n, t, need, last)
            last = need
    for t in (100, 255, 512, 1024, 1025, 4096, 16384, pick(200000)):                    # along the sequences
        last = 0
        for n in range(1, 600):
            need = size(n, t)
            assert need >= last, (n, t, need, last)
            last = need


def test_stated_cases():
    """One prompt a token longer, one sequence more of the same tokens, gradients of a few tokens more."""
    size = lambda n, t, back=False: K.kda_ssm_chunk_workspace_size(n, t, 32, 1, 128, 64, bf, back)   # noqa: E731
    assert size(1, 12288) <= size(1, 12289) <= size(1, 14000)
    assert size(15, 16384) <= size(16, 16384)
    assert size(1, 16320, True) <= size(1, 16384, True)


def test_costs_little():
    """What the bound asks for beyond the parts that a call lays out: no workspace where nothing so small ever needs one,
    less than 64 MB for segments, and in the gradients not a quarter more than the states of all chunks."""
    for H, G, dk, dv in HEADS:
        for n, t in ((1, 100), (300, 255), (7, 0)):
            assert K.kda_ssm_chunk_workspace_size(n, t, H, G, dk, dv, bf) == 0
        for n, t in ((1, 65536), (16, 16384), (200, 60000)):
            assert K.kda_ssm_chunk_workspace_size(n, t, H, G, dk, dv, bf) < 64 << 20
    states = (4 * 4096 // 64 + 4) * 32 * 128 * 64 * 8
    assert K.kda_ssm_chunk_workspace_size(4, 4 * 4096, 32, 1, 128, 64, bf, True) < 1.25 * states


def test_out_of_range():
    """Sizes beyond what the convolution's gradients take: 0, not what is left of a product past 64 bits."""
    for T, C in ((1 << 31, 64), (1 << 62, 64), (1, (1 << 23) + 1), (1 << 30, (1 << 31) - 1)):
        assert K.kda_conv_bwd_workspace_size(1, T, C, 4) == 0, (T, C)
    assert K.kda_conv_bwd_workspace_size(1, (1 << 31) - 1, 1 << 23, 4) > 1 << 40


def test_other_calls_never_fall():
    """The convolution's gradients and the slot pools: the same holds."""
    r = random.Random(2)
    for _ in range(20000):
        n, t, C = r.randrange(1, 400), int(200000 ** r.random()), r.choice([1, 64, 4352])
        for m, u in ((n + r.randrange(3), t), (n, t + r.randrange(200))):
            assert K.kda_conv_bwd_workspace_size(m, u, C, 4) >= K.kda_conv_bwd_workspace_size(n, t, C, 4), (n, t, m, u)
            assert K.kda_slots_workspace_size(n + m, u) >= K.kda_slots_workspace_size(n, t)
