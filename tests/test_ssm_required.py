"""Tensors that a convolution, scan or slot call cannot do without: the binding refuses None by name, before anything
else is asked of it (CPU)."""
import pytest
import torch

from gated_delta_rule_60_amd import kda as K

i32 = torch.int32


def conv():
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    return {"kda_conv_fwd": (K.kda_conv_fwd, dict(x=x, weight=w)),
            "kda_conv_bwd": (K.kda_conv_bwd, dict(x=x, weight=w, dy=x)),
            "kda_conv_step": (K.kda_conv_step, dict(x=x[0], weight=w, windows=torch.zeros(5, 3, 8)))}


def scan():
    x, dt, A, B = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 4), torch.zeros(4), torch.zeros(2, 5, 2, 64)
    prompt = dict(x=x, dt=dt, A=A, B=B, C=B)
    token = dict(x=x[0], dt=dt[0], A=A, B=B[0], C=B[0], state=torch.zeros(5, 4, 64, 64))
    return {"kda_ssm_chunk_fwd": (K.kda_ssm_chunk_fwd, prompt), "kda_ssm_chunk_bwd": (K.kda_ssm_chunk_bwd, dict(prompt, dy=x)),
            "kda_ssm_decode_step": (K.kda_ssm_decode_step, token)}


def slots():
    refs = torch.zeros(6, dtype=i32)
    pool = dict(pool=torch.zeros(6, 3), refs=refs)
    return {"kda_slots_retain": (K.kda_slots_retain, dict(refs=refs, slots=refs)),
            "kda_slots_release": (K.kda_slots_release, dict(refs=refs, slots=refs)),
            "kda_slots_fork": (K.kda_slots_fork, dict(pool, parents=refs)), "kda_slots_compact": (K.kda_slots_compact, pool)}


CALLS = {**conv(), **scan(), **slots()}


@pytest.mark.parametrize("fn,name", [(fn, name) for fn, (_, args) in CALLS.items() for name in args if name != "pool"])
@pytest.mark.parametrize("value", [None, 1.0])
def test_refused_by_name(fn, name, value):
    call, args = CALLS[fn]
    with pytest.raises((TypeError, ValueError), match=rf"^{fn}: {name} must be "):
        call(**{**args, name: value})


@pytest.mark.parametrize("count", [-1, 1 << 31, 1.5, None])
def test_number_of_new_sequences(count):
    """A number of new sequences that the call cannot carry out is refused as such, not by what it would allocate."""
    refs = torch.zeros(6, dtype=i32)
    with pytest.raises((TypeError, ValueError), match="^kda_slots_fork: parents must be "):
        K.kda_slots_fork(torch.zeros(6, 3), refs, count)
