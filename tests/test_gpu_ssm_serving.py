"""Decode steps of the scan, and convolution, scan, state cache and slots as a layer would use them together."""
import pytest
import torch

import ssm_ref as R
from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV
from test_gpu_ssm import check, make

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def token(d, t):
    return [d[k][:, t] for k in ("x", "dt")] + [d["A"]] + [d[k][:, t] for k in ("B", "C")]


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("y_dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_steps(dtype, y_dtype, dk, dv):
    """Tokens one by one, states in slots in any order, against the reference."""
    d = make(dtype, [5, 5, 5], H=6, G=2, dk=dk, dv=dv, packed=False, state=True)
    slots = torch.tensor([3, 0, 5], dtype=torch.int32, device=DEV)
    pool = torch.full((6, 6, dk, dv), 2.5, device=DEV)
    pool[slots.long()] = d["h0"]
    y = torch.stack([K.kda_ssm_decode_step(*token(d, t), pool, D=d["D"], dt_bias=d["bias"], slots=slots, y_dtype=y_dtype)
                     for t in range(5)], 1)
    torch.cuda.synchronize()
    mag = {k: (v.abs() if isinstance(v, torch.Tensor) and k not in ("dt", "A", "bias") else v) for k, v in d["ref"].items()}
    (y_ref, h_ref), (y_mag, h_mag) = R.scan(**d["ref"]), R.scan(**mag)
    check("y", y, y_ref, y_mag, f32)          # no bf16 terms in a step: fp32 accuracy
    check("state", pool[slots.long()], h_ref, h_mag, f32)
    assert (pool[[1, 2, 4]] == 2.5).all()


def test_step_options_and_slots():
    """No D, no bias, no slots; skipped and repeated slots; N = 0."""
    d = make(f32, [1, 1, 1, 1, 1], H=4, G=1, dk=64, dv=64, packed=False, state=True, skip=False, bias=False)
    a = d["h0"].clone()
    ya = K.kda_ssm_decode_step(*token(d, 0), a)
    y_ref, h_ref = R.scan(**d["ref"])
    assert (ya.double().cpu() - y_ref[:, 0]).abs().max() < 1e-4 and (a.double().cpu() - h_ref).abs().max() < 1e-4
    pool = d["h0"].clone()
    slots = torch.tensor([1, -1, 4, 1, 5], dtype=torch.int32, device=DEV)
    y = K.kda_ssm_decode_step(*token(d, 0), pool, slots=slots)
    two = d["h0"][[4, 1]].contiguous()
    want = K.kda_ssm_decode_step(*[t if t is d["A"] else t[[2, 3]].contiguous() for t in token(d, 0)], two)
    torch.cuda.synchronize()
    assert torch.equal(y[[2, 3]], want) and (y[[0, 1, 4]] == 0).all()
    assert torch.equal(pool[[4, 1]], two) and torch.equal(pool[[0, 2, 3]], d["h0"][[0, 2, 3]])
    none = [t if t is d["A"] else t[:0] for t in token(d, 0)]
    assert K.kda_ssm_decode_step(*none, pool).shape == (0, 4, 64)


def test_long_decode_keeps_its_accuracy():
    """A thousand steps with one and the same decay: its rounding must not add up."""
    H, dk, dv, n = 2, 64, 64, 1000
    g = torch.Generator().manual_seed(0)
    x, B, C = torch.randn(1, H, dv, generator=g).to(DEV), torch.randn(1, 1, dk, generator=g).to(DEV), torch.randn(1, 1, dk, generator=g).to(DEV)
    dt, A = torch.full((1, H), -4.0, device=DEV), torch.tensor([-0.05, -0.5], device=DEV)
    S = torch.randn(1, H, dk, dv, generator=g).to(DEV)
    ref = S.double()
    delta = torch.log1p(torch.exp(dt.double()))
    step = (delta[0, :, None, None] * B.double()[0, 0, :, None] * x.double()[0, :, None, :])
    a = torch.exp(delta * A.double())[0, :, None, None]
    for _ in range(n):
        K.kda_ssm_decode_step(x, dt, A, B, C, S)
        ref = ref * a + step
    # n roundings of 2^-24 each, of either sign, and delta's few ulps times the log-decay kept (below 1/2)
    err = ((S.double() - ref).pow(2).mean() / ref.pow(2).mean()).sqrt().item()
    assert err < 2e-6, err


def test_layer_serves_prompts_then_tokens():
    """A layer's convolution and scan over packed prompts, the states kept in slots, requests forked, released and moved,
    then tokens: equal to the same sequences run as one prompt each, for states and windows, and near for outputs."""
    H, G, dk, dv, W = 4, 2, 64, 64, 4
    row = H * dv + 2 * G * dk
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g)
    w, b = r(row, W).to(DEV) / 2, 0.1 * r(row).to(DEV)
    A, bias, D = (-0.5 - torch.rand(H, generator=g)).to(DEV), (r(H) - 2).to(DEV), r(H).to(DEV)
    lens = [70, 3, 130]
    n_tok = 6
    # the children of requests 0 and 2 go on with tokens of their own
    prompts = [r(n, row) for n in lens]
    tails = [r(n_tok, row) for _ in range(4)]
    dts = [r(n, H) for n in lens]
    dt_tails = [r(n_tok, H) for _ in range(4)]

    def split(u):
        return (u[..., :H * dv].unflatten(-1, (H, dv)), u[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk)),
                u[..., H * dv + G * dk:].unflatten(-1, (G, dk)))

    def prompt(u, dt, cu=None):
        u, win = K.kda_conv_fwd(u.to(DEV), w, b, cu_seqlens=cu, output_final_state=True)
        x, B, C = split(u)
        y, S = K.kda_ssm_chunk_fwd(x, dt.to(DEV), A, B, C, D=D, dt_bias=bias, cu_seqlens=cu)
        return y, S, win

    cu = torch.tensor([0, 70, 73, 203], dtype=torch.int32, device=DEV)
    _, S, win = prompt(torch.cat(prompts)[None], torch.cat(dts)[None], cu)
    pool = [torch.full((10, H, dk, dv), 5.0, device=DEV), torch.full((10, W - 1, row), 5.0, device=DEV)]
    refs = torch.zeros(10, dtype=torch.int32, device=DEV)
    refs[[0, 1, 4]] = 1                                   # other requests
    slots = K.kda_slots_fork(pool, refs, 3)
    assert slots.tolist() == [2, 3, 5]
    K.kda_slots_copy([S, win], pool, dst_slots=slots)
    kids = K.kda_slots_fork(pool, refs, slots[[0, 2]].contiguous())
    K.kda_slots_release(refs, torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV))
    table = torch.cat([slots, kids])
    used = K.kda_slots_compact(pool, refs, table)
    assert used.item() == 5 and table.tolist()[1] == -1   # request 1 has ended
    live = table[[0, 2, 3, 4]].contiguous()
    outs = []
    for t in range(n_tok):
        u = K.kda_conv_step(torch.stack([x[t] for x in tails]).to(DEV), w, pool[1], b, slots=live)
        x, B, C = split(u)
        outs.append(K.kda_ssm_decode_step(x, torch.stack([x[t] for x in dt_tails]).to(DEV), A, B, C, pool[0], D=D,
                                          dt_bias=bias, slots=live))
    torch.cuda.synchronize()
    for i, of in enumerate([0, 2, 0, 2]):
        y, S1, w1 = prompt(torch.cat([prompts[of], tails[i]])[None], torch.cat([dts[of], dt_tails[i]])[None])
        got = torch.stack([o[i] for o in outs])
        assert torch.equal(pool[1][live[i].item()], w1[0])
        # both sides are fp32 results of the same sums: 2^-15 of the largest each
        assert (got - y[0, -n_tok:]).abs().max() <= 2.0 ** -14 * y.abs().max()
        assert (pool[0][live[i].item()] - S1[0]).abs().max() <= 2.0 ** -14 * S1.abs().max()


def test_states_through_the_8_bit_cache():
    """A prefix's final state parked as 8-bit codes, its slot forked with codes and scales, picked up again."""
    H, dk, dv = 4, 128, 64
    d = make(bf, [200], H, 1, dk, dv, packed=False, state=False)
    _, S = K.kda_ssm_chunk_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"])
    codes = torch.zeros(5, H, dk, dv, dtype=torch.int8, device=DEV)
    scales = torch.zeros(5, H, dk, dv // 32, device=DEV)
    refs = torch.zeros(5, dtype=torch.int32, device=DEV)
    slot = K.kda_slots_fork([codes, scales], refs, 1)
    K.kda_state_store(S, codes, scales, slot)
    kids = K.kda_slots_fork([codes, scales], refs, slot)
    back = K.kda_state_load(codes, scales, torch.cat([slot, kids]))
    torch.cuda.synchronize()
    assert kids.tolist() == [1] and torch.equal(back[0], back[1])
    step = S.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 127
    assert ((back[:1] - S).unflatten(-1, (-1, 32)).abs() <= 0.5001 * step).all()


def _layer(d, pool, slots):
    y, S = K.kda_ssm_chunk_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"], initial_state=d["h0"])
    g = K.kda_ssm_chunk_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], D=d["D"], dt_bias=d["bias"],
                            initial_state=d["h0"], d_final_state=d["dhT"])
    row = d["row_dev"]
    u, win = K.kda_conv_fwd(row, d["w"], output_final_state=True)
    du = K.kda_conv_bwd(row, d["w"], u)
    step = K.kda_ssm_decode_step(*token(d, 0), pool, D=d["D"], dt_bias=d["bias"], slots=slots)
    return [y, S, u, win, step] + [t for t in g + du if t is not None]


def _setup(seed=0):
    d = make(bf, [700, 700], H=4, G=1, dk=64, dv=64, packed=False, state=True, seed=seed)
    d["row_dev"] = d["row"].to(DEV)
    d["w"] = torch.randn(d["row"].shape[-1], 4, generator=torch.Generator().manual_seed(seed)).to(DEV)
    return d


def test_another_stream():
    d = _setup()
    slots = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    want = _layer(d, d["h0"].clone(), slots)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    pool = d["h0"].clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _layer(d, pool, slots)
    y, _ = K.kda_ssm_chunk_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"], initial_state=d["h0"],
                               stream=s.cuda_stream)
    s.synchronize()
    for a, b in zip(want + [want[0]], got + [y]):
        assert torch.equal(a, b)


def test_captured_and_replayed():
    """All of a layer's calls in one captured graph, replayed on new inputs with eager work in between."""
    d = _setup()
    slots = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    pool = d["h0"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _layer(d, pool, slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = _layer(d, pool, slots)
    for seed in (1, 2, 3):
        e = _setup(seed)
        d["x"]._base.copy_(e["x"]._base)                # the row buffer that x, B and C are parts of
        for k in ("dt", "A", "D", "bias", "h0", "dy", "dhT", "row_dev", "w"):
            d[k].copy_(e[k])
        pool.copy_(e["h0"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = _layer(e, e["h0"].clone(), slots)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
