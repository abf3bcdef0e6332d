"""GPU parity of linear attention with one decay per head (prefill, gradients, decode step) with the
plain fp64 recurrences of linear_ref.py.

Tolerances are elementwise.  With M the sum of the magnitudes of everything an element adds up
(linear_ref.*_abs) and u = 2^-24:
  * an element of o, dq, dk or dv is a sum over up to dk (dv) state channels and 64 tokens of a
    chunk, each rounded a few times, of a state that has itself been rounded at most about twice per
    token: (2 T + 3 * 128 + 3 * 64 + 64) u M = (2 T + 640) u M;
  * bf16 inputs: states and decayed scores enter the products as two bf16 terms, each value off by
    at most 2^-8 * 2^-8 of itself: 2^-16 M more, and 2^-16 M again for a score formed of such terms;
  * a state element: (2 T + 640) u M;
  * an output's own rounding: half a step, eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

import linear_ref as R
from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
DECAYS = [-0.3, 0.0, -1e-3, -5.0, float("-inf"), -0.02, -40.0, -1e-5]


def make(B, T, H, dk, dv, dtype, lens=None, state=True, seed=0, zero_norm=False):
    gen = torch.Generator("cpu").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)                                  # noqa: E731
    cu = None
    if lens is not None:
        B, T = 1, sum(lens)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    N = B if lens is None else len(lens)
    d = dict(q=rn(B, T, H, dk), k=rn(B, T, H, dk), v=rn(B, T, H, dv), do=rn(B, T, H, dv))
    d = {n: (x / (dk if n in "qk" else 1) ** 0.5).to(dtype) for n, x in d.items()}
    d.update(g=torch.tensor((DECAYS * (H // len(DECAYS) + 1))[:H]),
             h0=rn(N, H, dk, dv) if state else None, dhT=rn(N, H, dk, dv) if state else None, cu=cu)
    return d


def dev(x):
    return None if x is None else x.to(DEV)


def host64(d, *names):
    return [R.np64(d[n]) for n in names]


def longest(d):
    return int((d["cu"][1:] - d["cu"][:-1]).max()) if d["cu"] is not None else d["q"].shape[1]


def close(got, ref, mag, terms, dtype, what):
    tol = terms * mag + np.abs(ref) * (torch.finfo(dtype).eps / 2) * 1.01 + 1e-37
    got = R.np64(got)
    assert np.isfinite(got).all(), what
    worst = float((np.abs(got - ref) / tol).max()) if got.size else 0.0
    say(f"  {what}: worst {worst:.3f} of the tolerance")
    assert worst <= 1.0, what


def terms(d, out=True):
    t = (2 * longest(d) + 640) * U
    return t + 2 * 2.0 ** -16 if out and d["q"].dtype == BF else t


def check_fwd(d, scale=1.0, o_dtype=None, **kw):
    q, k, v, g, h0 = host64(d, "q", "k", "v", "g", "h0")
    ref = R.forward(q, k, v, g, h0, d["cu"], scale)
    mag = R.forward_abs(q, k, v, g, h0, d["cu"], scale)
    o, hT = K.kda_linear_chunk_fwd(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["g"]),
                                   initial_state=dev(d["h0"]), cu_seqlens=dev(d["cu"]),
                                   scale=scale, o_dtype=o_dtype, **kw)
    torch.cuda.synchronize()
    close(o, ref[0], mag[0], terms(d), o.dtype, "o")
    close(hT, ref[1], mag[1], terms(d, False), F32, "final state")


def check_bwd(d, scale=1.0, want_dh0=True):
    x = host64(d, "q", "k", "v", "g", "do", "h0", "dhT")
    ref = R.backward(*x, d["cu"], scale)
    mag = R.backward_abs(*x, d["cu"], scale)
    got = K.kda_linear_chunk_bwd(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["g"]), dev(d["do"]),
                                 initial_state=dev(d["h0"]), d_final_state=dev(d["dhT"]),
                                 cu_seqlens=dev(d["cu"]), scale=scale,
                                 output_d_initial_state=want_dh0)
    torch.cuda.synchronize()
    for i, name in enumerate(("dq", "dk", "dv")):
        close(got[i], ref[i], mag[i], terms(d), got[i].dtype, name)
    if want_dh0:
        close(got[3], ref[3], mag[3], terms(d, False), F32, "d_initial_state")
    else:
        assert got[3] is None


SIZES = [(128, 128), (64, 64), (64, 128), (128, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 129, 200])
def test_prefill_lengths(T, dk, dv, dtype):
    check_fwd(make(2, T, 3, dk, dv, dtype, seed=T))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 129, 200])
def test_gradient_lengths(T, dk, dv, dtype):
    check_bwd(make(2, T, 3, dk, dv, dtype, seed=100 + T))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_decay_scale_and_output_type(dtype):
    d = make(1, 150, 8, 64, 128, dtype, seed=5)
    check_fwd(d, scale=-0.37)
    check_fwd(d, scale=2.5, o_dtype=F32)
    check_fwd(d, o_dtype=BF)
    check_bwd(d, scale=-0.37)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_states(dtype):
    d = make(2, 97, 3, 128, 64, dtype, state=False, seed=6)
    check_fwd(d)
    check_bwd(d)
    check_bwd(d, want_dh0=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[0, 1, 64, 0, 65, 130, 0], [0], [1], [333, 0, 5], [64, 64, 64],
                                  [7] * 20])
def test_packed(lens, dtype):
    d = make(1, 0, 3, 128, 128, dtype, lens=lens, seed=sum(lens))
    check_fwd(d)
    check_bwd(d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [dict(B=1, T=2500), dict(B=1, T=0, lens=[1500, 3, 0, 1111])])
def test_long_sequences(shape, dtype):
    """Long enough, with few enough heads, that one sequence's tokens are worked on in parallel."""
    d = make(H=2, dk=128, dv=128, dtype=dtype, seed=9, **shape)
    d["g"] = torch.tensor([-1e-3, -0.05])
    check_fwd(d)
    check_bwd(d)


def test_full_size_sampled_heads():
    """4 x 4096 tokens x 16 heads: two (sequence, head) units against the fp64 recurrence."""
    d = make(4, 4096, 16, 128, 128, BF, seed=11)
    d["g"] = -torch.exp2(-1.0 - 10.0 * torch.arange(16) / 16)
    o, hT = K.kda_linear_chunk_fwd(*(dev(d[n]) for n in ("q", "k", "v", "g", "h0")))
    grads = K.kda_linear_chunk_bwd(*(dev(d[n]) for n in ("q", "k", "v", "g", "do", "h0", "dhT")))
    torch.cuda.synchronize()
    for n, h in ((0, 15), (3, 6)):
        s = dict(cu=None, g=d["g"][h:h + 1])
        for name in ("q", "k", "v", "do"):
            s[name] = d[name][n:n + 1, :, h:h + 1]
        for name in ("h0", "dhT"):
            s[name] = d[name][n:n + 1, h:h + 1]
        x = host64(s, "q", "k", "v", "g", "h0")
        ref, mag = R.forward(*x), R.forward_abs(*x)
        close(o[n:n + 1, :, h:h + 1], ref[0], mag[0], terms(s), BF, "o")
        close(hT[n:n + 1, h:h + 1], ref[1], mag[1], terms(s, False), F32, "final state")
        x = host64(s, "q", "k", "v", "g", "do", "h0", "dhT")
        ref, mag = R.backward(*x), R.backward_abs(*x)
        for i, name in enumerate(("dq", "dk", "dv")):
            close(grads[i][n:n + 1, :, h:h + 1], ref[i], mag[i], terms(s), BF, name)
        close(grads[3][n:n + 1, h:h + 1], ref[3], mag[3], terms(s, False), F32, "d_initial_state")


def test_gradients_against_differences():
    """fp32: <do, o(x + e) - o(x - e)> / 2 + <dhT, same of hT> equals <dx, e>; the outputs are linear
    in each input, so the step may be large and the difference has no error of its own."""
    d = make(2, 100, 3, 64, 64, F32, seed=12)
    x = {n: dev(d[n]) for n in ("q", "k", "v", "g", "do", "h0", "dhT")}
    grads = dict(zip(("q", "k", "v", "h0"), K.kda_linear_chunk_bwd(
        x["q"], x["k"], x["v"], x["g"], x["do"], initial_state=x["h0"], d_final_state=x["dhT"])))

    def loss(**over):
        y = {**x, **over}
        o, hT = K.kda_linear_chunk_fwd(y["q"], y["k"], y["v"], y["g"], initial_state=y["h0"])
        return (o.double() * x["do"].double()).sum() + (hT.double() * x["dhT"].double()).sum()

    gen = torch.Generator("cpu").manual_seed(3)
    mag = R.backward_abs(*host64(d, "q", "k", "v", "g", "do", "h0", "dhT"))
    for i, name in enumerate(("q", "k", "v", "h0")):
        e = torch.randn(x[name].shape, generator=gen)
        diff = float(loss(**{name: x[name] + dev(e)}) - loss(**{name: x[name] - dev(e)})) / 2
        dot = float((grads[name].double().cpu() * e.double()).sum())
        # x +- e is rounded to fp32 (half a step of a value of up to about |x| + |e|), and every
        # product on both sides as in the module's tolerances
        size = float((mag[i] * (np.abs(R.np64(x[name])) + np.abs(e.numpy()))).sum())
        say(f"  {name}: {diff:.9g} {dot:.9g}")
        assert abs(diff - dot) <= (2 * 100 + 640) * U * size * 2, name


def test_in_place_state_and_zero_tokens():
    d = make(2, 130, 3, 128, 128, BF, seed=13)
    a = [dev(d[n]) for n in ("q", "k", "v", "g")]
    o, hT = K.kda_linear_chunk_fwd(*a, initial_state=dev(d["h0"]))
    S = dev(d["h0"])
    o2, S2 = K.kda_linear_chunk_fwd(*a, initial_state=S, final_state=S)
    assert S2 is S and torch.equal(o, o2) and torch.equal(S, hT)
    e = [x[:, :0].contiguous() for x in a[:3]]
    o0, h0 = K.kda_linear_chunk_fwd(*e, a[3], initial_state=dev(d["h0"]))
    assert o0.numel() == 0 and torch.equal(h0, dev(d["h0"]))
    o0, h0 = K.kda_linear_chunk_fwd(*e, a[3])
    assert torch.equal(h0, torch.zeros_like(h0))
    _, _, _, dh = K.kda_linear_chunk_bwd(*e, a[3], o0, d_final_state=dev(d["dhT"]),
                                         output_d_initial_state=True)
    assert torch.equal(dh, dev(d["dhT"]))
    _, none = K.kda_linear_chunk_fwd(*a, output_final_state=False)
    assert none is None


@pytest.mark.parametrize("shape", [dict(B=1, T=2500), dict(B=1, T=0, lens=[1500, 3, 0, 1111])])
def test_in_place_state_of_a_long_sequence(shape):
    """The segments of a sequence run at the same time: the last one's final state must not overwrite the
    initial state that the first one starts from."""
    d = make(H=2, dk=128, dv=128, dtype=BF, seed=16, **shape)
    d["g"] = torch.tensor([-1e-3, -0.05])
    a = [dev(d[n]) for n in ("q", "k", "v", "g")]
    o, hT = K.kda_linear_chunk_fwd(*a, initial_state=dev(d["h0"]), cu_seqlens=dev(d["cu"]))
    for _ in range(3):
        S = dev(d["h0"])
        o2, _ = K.kda_linear_chunk_fwd(*a, initial_state=S, final_state=S, cu_seqlens=dev(d["cu"]))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, hT)


def test_debug_validation(monkeypatch):
    """KDA_DEBUG_VALIDATE refuses positive or NaN decays and malformed offsets, and takes -inf."""
    d = make(1, 0, 2, 64, 64, BF, lens=[70, 30], seed=32)
    q, k, v, do = (dev(d[n]) for n in ("q", "k", "v", "do"))
    S = torch.zeros((1, 2, 64, 64), device=DEV)
    one = [x[0, :1].contiguous() for x in (q, k, v)]
    monkeypatch.setenv("KDA_DEBUG_VALIDATE", "1")
    good = torch.tensor([-0.1, float("-inf")], device=DEV)
    K.kda_linear_chunk_fwd(q, k, v, good, cu_seqlens=dev(d["cu"]))
    K.kda_linear_decode_step(*one, good, S)
    for bad in (0.25, float("nan")):
        g = torch.tensor([-0.1, bad], device=DEV)
        for call in (lambda: K.kda_linear_chunk_fwd(q, k, v, g), lambda: K.kda_linear_chunk_bwd(q, k, v, g, do),
                     lambda: K.kda_linear_decode_step(*one, g, S)):
            with pytest.raises(K.KDAError) as e:
                call()
            assert e.value.status == 1
    for cu in ([0, 80, 60], [1, 70, 100], [0, 70, 99]):
        with pytest.raises(K.KDAError) as e:
            K.kda_linear_chunk_fwd(q, k, v, good, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert e.value.status == 1


def test_split_prefill_continues():
    """Two prefills, the second from the first one's state, against one."""
    d = make(1, 300, 2, 128, 128, F32, seed=14)
    cut = lambda lo, hi: [dev(d[n][:, lo:hi].contiguous()) for n in ("q", "k", "v")]   # noqa: E731
    g = dev(d["g"])
    o, hT = K.kda_linear_chunk_fwd(*cut(0, 300), g, initial_state=dev(d["h0"]))
    o1, S = K.kda_linear_chunk_fwd(*cut(0, 101), g, initial_state=dev(d["h0"]))
    o2, S = K.kda_linear_chunk_fwd(*cut(101, 300), g, initial_state=S)
    mag = R.forward_abs(*host64(d, "q", "k", "v", "g", "h0"))
    close(torch.cat([o1, o2], 1), R.np64(o), mag[0], 2 * terms(d), F32, "o")
    close(S, R.np64(hT), mag[1], 2 * terms(d, False), F32, "state")


def test_deterministic_and_bf16_output_rounding():
    d = make(2, 1000, 4, 128, 128, BF, seed=15)
    a = [dev(d[n]) for n in ("q", "k", "v", "g", "h0")]
    o32, h1 = K.kda_linear_chunk_fwd(*a, o_dtype=F32)
    o16, h2 = K.kda_linear_chunk_fwd(*a)
    o16b, h3 = K.kda_linear_chunk_fwd(*a)
    assert torch.equal(o32.to(BF), o16) and torch.equal(o16, o16b)
    assert torch.equal(h1, h2) and torch.equal(h1, h3)
    b = a[:4] + [dev(d["do"])]
    g1 = K.kda_linear_chunk_bwd(*b, initial_state=a[4], d_final_state=dev(d["dhT"]))
    g2 = K.kda_linear_chunk_bwd(*b, initial_state=a[4], d_final_state=dev(d["dhT"]))
    assert all(torch.equal(x, y) for x, y in zip(g1, g2))


# ------------------------------------------------------------------------------------ decode

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("N,H", [(1, 1), (5, 8), (33, 3)])
def test_decode_steps(N, H, dk, dv, dtype):
    steps = 3
    d = make(N, steps, H, dk, dv, dtype, seed=20 + N)
    x = host64(d, "q", "k", "v", "g", "h0")
    ref, mag = R.forward(*x, None, 0.5), R.forward_abs(*x, None, 0.5)
    S = dev(d["h0"])
    o = [K.kda_linear_decode_step(*(dev(d[n][:, t].contiguous()) for n in "qkv"), dev(d["g"]), S,
                                  scale=0.5, o_dtype=F32) for t in range(steps)]
    o16 = K.kda_linear_decode_step(*(dev(d[n][:, 0].contiguous()) for n in "qkv"), dev(d["g"]),
                                   dev(d["h0"]), scale=0.5, o_dtype=BF)
    torch.cuda.synchronize()
    t = (2 * steps + 640) * U                       # fp32 arithmetic throughout
    close(torch.stack(o, 1), ref[0], mag[0], t, F32, "o")
    close(S, ref[1], mag[1], t, F32, "state")
    assert torch.equal(o16, o[0].to(BF))


def test_decode_no_sequences():
    z = torch.zeros((0, 2, 64), device=DEV)
    o = K.kda_linear_decode_step(z, z, z, torch.zeros(2, device=DEV),
                                 torch.zeros((0, 2, 64, 64), device=DEV))
    assert o.shape == (0, 2, 64)


# ------------------------------------------------------------------------------------ streams

def _pass(d, S, outs):
    """A prefill, its gradients and a decode step into given buffers, on the current stream."""
    K.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                           final_state=outs["hT"], o=outs["o"], workspace=outs["ws"])
    K.kda_linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["h0"],
                           d_final_state=d["dhT"], dq=outs["dq"], dk=outs["dk"], dv=outs["dv"],
                           d_initial_state=outs["dh0"], workspace=outs["wsb"])
    S.copy_(outs["hT"])
    K.kda_linear_decode_step(*(d[n][:, 0].contiguous() for n in "qkv"), d["g"], S, o=outs["od"])


def _buffers(d):
    B, T, H, dk = d["q"].shape
    dv = d["v"].shape[-1]
    mk = lambda s, t=BF: torch.full(s, float("nan"), dtype=t, device=DEV)      # noqa: E731
    ws = lambda b: torch.empty(max(16, K.kda_linear_chunk_workspace_size(B, B * T, H, dk, dv,   # noqa: E731
                                                                         BF, b)), dtype=torch.uint8, device=DEV)
    return dict(o=mk(d["v"].shape), hT=mk(d["h0"].shape, F32), dq=mk(d["q"].shape), dk=mk(d["k"].shape),
                dv=mk(d["v"].shape), dh0=mk(d["h0"].shape, F32), od=mk((B, H, dv)), ws=ws(False), wsb=ws(True))


@pytest.mark.parametrize("T", [130, 2100])
def test_other_stream_and_captured_replays(T):
    d = {n: dev(x) for n, x in make(1, T, 2, 128, 128, BF, seed=30).items()}
    want, S = _buffers(d), torch.empty_like(d["h0"])
    _pass(d, S, want)
    torch.cuda.synchronize()
    names = [n for n in want if not n.startswith("ws")]
    side = torch.cuda.Stream()
    got = _buffers(d)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _pass(d, S, got)
    side.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in names)
    graph = torch.cuda.CUDAGraph()
    got = _buffers(d)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _pass(d, S, got)
    for _ in range(3):
        for n in names:
            got[n].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], got[n]) for n in names)
        _pass(d, S, _buffers(d))                 # the program's own work between the replays
        torch.cuda.synchronize()


def test_two_calls_at_once():
    """Prefills and gradients of two inputs on two streams, each with workspaces of its own."""
    ds = [{n: dev(x) for n, x in make(1, T, 2, 128, 128, BF, seed=40 + T).items()} for T in (2100, 1500)]
    want = [_buffers(d) for d in ds]
    for d, b in zip(ds, want):
        _pass(d, torch.empty_like(d["h0"]), b)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ds], [_buffers(d) for d in ds]
    states = [torch.empty_like(d["h0"]) for d in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, d, S, b in zip(streams, ds, states, got):
            with torch.cuda.stream(st):
                _pass(d, S, b)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[n], b[n]) for n in a if not n.startswith("ws"))


def test_tensors_beyond_four_gigabytes():
    """One sequence of 2^20 + 5000 tokens x 17 heads (4.6 GB per tensor) under a decay that forgets within
    some hundred tokens: its last 4096 tokens against a call on them alone, where 1024 tokens in nothing of
    what came before is left (e^(-0.5 * 1024)).  Both results round the same numbers, so they differ by a
    half step of each and by the roundings on the way: sums of at most 1 / (1 - e^-0.5) < 2.6 terms of
    |q.k| <= 1 times |v| < 7, each within (2 * 256 + 640) 2^-24 + 2 * 2^-16 of itself."""
    T, H, tail, skip = (1 << 20) + 5000, 17, 4096, 1024
    gen = torch.Generator(DEV).manual_seed(50)

    def unit():
        x = torch.randn((1, T, H, 128), generator=gen, device=DEV, dtype=BF)
        for i in range(0, T, 1 << 17):
            part = x[:, i:i + (1 << 17)].float()
            x[:, i:i + (1 << 17)] = part / part.norm(dim=-1, keepdim=True)
        return x
    q, k = unit(), unit()
    v, do = (torch.randn((1, T, H, 128), generator=gen, device=DEV, dtype=BF) for _ in range(2))
    g = torch.full((H,), -0.5, device=DEV)
    cut = lambda x: x[:, T - tail:].contiguous()                                   # noqa: E731
    # q and k are rounded to bf16 after normalising: |q.k| <= 1 + 2^-6
    slack = 2 * 2.6 * 1.02 * 7 * ((2 * 256 + 640) * U + 2 * 2.0 ** -16)

    def same(a, b, lo):
        a, b = a[:, lo:].float(), b[:, lo:].float()
        assert bool(((a - b).abs() <= slack + 2 * 2.0 ** -8 * torch.maximum(a.abs(), b.abs())).all())
    o, S = K.kda_linear_chunk_fwd(q, k, v, g)
    o1, S1 = K.kda_linear_chunk_fwd(cut(q), cut(k), cut(v), g)
    same(cut(o), o1, skip)
    assert float((S - S1).abs().max()) <= slack
    del o
    grads = K.kda_linear_chunk_bwd(q, k, v, g, do)
    # |do| has 128 elements: dq, dk sum |v.do| <= |v| |do| < 16^2 of unit vectors' elements
    slack *= 16 * 16 / 7
    for x, y, lo in zip(grads, K.kda_linear_chunk_bwd(*(cut(x) for x in (q, k, v)), g, cut(do)), (skip, 0, 0)):
        same(cut(x), y, lo)


def test_rows_behind_the_sequences_stay():
    """A packed batch whose offsets end before T (malformed, but in bounds): nothing behind the last
    sequence is written."""
    d = make(1, 0, 2, 64, 64, BF, lens=[70, 30], seed=31)
    pad = lambda x: torch.cat([x, torch.full_like(x[:, :20], 3.0)], 1).to(DEV)     # noqa: E731
    q, k, v, do = (pad(d[n]) for n in ("q", "k", "v", "do"))
    o = torch.full_like(v, 7.0)
    K.kda_linear_chunk_fwd(q, k, v, dev(d["g"]), cu_seqlens=dev(d["cu"]), o=o)
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    K.kda_linear_chunk_bwd(q, k, v, dev(d["g"]), do, cu_seqlens=dev(d["cu"]), dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    for x in (o, dq, dk, dv):
        assert bool((x[:, 100:] == 7.0).all()) and bool((x[:, :100] != 7.0).any())
