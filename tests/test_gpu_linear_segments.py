"""Sequences worked on in segments, at every head size: the shapes, scales, output types and absent states
that reach the segment states, their scan and the full pass differently."""
import numpy as np
import pytest
import torch

import linear_ref as R
from gated_delta_rule_60_amd import kda as K
from test_gpu_linear import BF, F32, SIZES, check_bwd, check_fwd, dev, host64, make

pytestmark = pytest.mark.gpu
SHAPES = [dict(B=1, T=1100), dict(B=1, T=0, lens=[1030, 3, 0, 150])]


def segmented(dk, dv, dtype, state=True, seed=60, **shape):
    d = make(H=2, dk=dk, dv=dv, dtype=dtype, state=state, seed=seed, **shape)
    d["g"] = torch.tensor([-1e-3, -0.05])
    N = 1 if d["cu"] is None else d["cu"].numel() - 1
    for back in (False, True):      # a workspace for fewer than two segments' states: none ran in segments
        assert K.kda_linear_chunk_workspace_size(N, d["q"].shape[1], 2, dk, dv, dtype, back) >= \
            2 * 2 * dk * dv * 4 * (1 + back)
    return d


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("shape", SHAPES)
def test_sizes_and_scale(shape, dk, dv, dtype):
    d = segmented(dk, dv, dtype, **shape)
    check_fwd(d, scale=-0.37)
    check_bwd(d, scale=-0.37)


@pytest.mark.parametrize("dtype,o_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("shape", SHAPES)
def test_other_output_type(shape, dk, dv, dtype, o_dtype):
    check_fwd(segmented(dk, dv, dtype, seed=61, **shape), scale=0.6, o_dtype=o_dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("shape", SHAPES)
def test_no_states(shape, dk, dv, dtype):
    d = segmented(dk, dv, dtype, state=False, seed=62, **shape)
    check_fwd(d)
    check_bwd(d)
    check_bwd(d, want_dh0=False)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_no_final_state(dk, dv):
    """o and the gradients of q, k, v do not depend on whether a state is handed out beyond their own
    rounding: without one the update's products take two terms."""
    d = segmented(dk, dv, BF, seed=63, **SHAPES[0])
    x = host64(d, "q", "k", "v", "g", "h0")
    ref, mag = R.forward(*x), R.forward_abs(*x)
    a = [dev(d[n]) for n in ("q", "k", "v", "g")]
    o, none = K.kda_linear_chunk_fwd(*a, initial_state=dev(d["h0"]), output_final_state=False, o_dtype=F32)
    torch.cuda.synchronize()
    # a value as two bf16 terms: 2^-16; three such factors (state or score, its parts, the update)
    tol = ((2 * 1100 + 640) * 2.0 ** -24 + 3 * 2.0 ** -16) * mag[0] + np.abs(ref[0]) * 2.0 ** -24
    assert none is None and np.all(np.abs(R.np64(o) - ref[0]) <= tol)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_in_place_state(dk, dv):
    for shape in SHAPES:
        d = segmented(dk, dv, BF, seed=64, **shape)
        a = [dev(d[n]) for n in ("q", "k", "v", "g")]
        o, hT = K.kda_linear_chunk_fwd(*a, initial_state=dev(d["h0"]), cu_seqlens=dev(d["cu"]))
        S = dev(d["h0"])
        o2, _ = K.kda_linear_chunk_fwd(*a, initial_state=S, final_state=S, cu_seqlens=dev(d["cu"]))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, hT)


def test_captured_gradients_of_unequal_sizes():
    """Two full-pass launches follow the scan; replayed three times with eager work between."""
    d = segmented(64, 128, BF, seed=65, **SHAPES[1])
    x = {n: dev(t) for n, t in d.items()}
    run = lambda: K.kda_linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], initial_state=x["h0"],   # noqa: E731
                                         d_final_state=x["dhT"], cu_seqlens=x["cu"])
    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        run()
        torch.cuda.synchronize()
