"""Refusals of the linear-attention and state-cache calls, in the C ABI and in the binding.  CPU only:
the pointers are never dereferenced, each call fails validation (or has nothing to do) before any
device work."""
import ctypes

import pytest
import torch

from gated_delta_rule_60_amd import kda as K

FAKE = 1 << 40
INV, UNS, WS = 1, 2, 3
Q, KK, V, G, O, H0, HT, CU, WSP, DO, DQ, DK, DV, DH = (FAKE + i * 0x10000000 for i in range(14))
bf, f32 = torch.bfloat16, torch.float32


def P(x):
    return ctypes.c_void_p(x) if x else None


@pytest.fixture(scope="module")
def lib():
    return K.load_library()


def fwd(lib, q=Q, k=KK, v=V, in_dt=1, g=G, h0=0, hT=0, cu=0, o=O, o_dt=1, B=1, T=128, N=1, H=2, dk=128,
        dv=128, scale=1.0, ws=WSP, ws_bytes=1 << 27):
    return lib.kda_linear_chunk_fwd(P(q), P(k), P(v), in_dt, P(g), P(h0), P(hT), P(cu), P(o), o_dt, B, T,
                                    N, H, dk, dv, scale, P(ws), ws_bytes, None)


def bwd(lib, q=Q, k=KK, v=V, in_dt=1, g=G, h0=0, cu=0, do=DO, dhT=0, dq=DQ, dk_=DK, dv_=DV, dh0=0, B=1,
        T=128, N=1, H=2, dk=128, dv=128, scale=1.0, ws=WSP, ws_bytes=1 << 27):
    return lib.kda_linear_chunk_bwd(P(q), P(k), P(v), in_dt, P(g), P(h0), P(cu), P(do), P(dhT), P(dq),
                                    P(dk_), P(dv_), P(dh0), B, T, N, H, dk, dv, scale, P(ws), ws_bytes,
                                    None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_shared_refusals(lib, call):
    for bad in (dict(in_dt=7), dict(B=0), dict(T=-1), dict(H=0), dict(N=2), dict(B=2, N=2, cu=CU),
                dict(q=0), dict(k=0), dict(v=0), dict(g=0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(ws=Q), dict(ws=G), dict(h0=H0, ws=H0),
                dict(cu=CU, N=3, ws=CU)):
        assert call(lib, **bad) == INV, bad
    for bad in (dict(dk=96), dict(dv=256), dict(q=Q + 2), dict(k=KK + 8), dict(v=V + 4), dict(g=G + 2),
                dict(h0=H0 + 8), dict(cu=CU + 1, N=3), dict(ws=WSP + 4), dict(H=1 << 22, T=0)):
        assert call(lib, **bad) == UNS, bad


def test_workspace_refused(lib):
    for call, back in ((fwd, False), (bwd, True)):
        for N, tok, H in ((1, 65536, 2), (1, 4096, 1), (1, 65536, 32)):
            need = K.kda_linear_chunk_workspace_size(N, tok, H, 128, 128, backward=back)
            if need:
                kw = dict(T=tok, H=H, k=Q + (1 << 34), v=Q + (2 << 34), o=Q + (3 << 34), do=Q + (4 << 34),
                          dq=Q + (5 << 34), dk_=Q + (6 << 34), dv_=Q + (7 << 34), g=Q + (8 << 34),
                          ws=Q + (9 << 34))
                for x in (("do", "dq", "dk_", "dv_") if call is fwd else ("o",)):
                    del kw[x]
                assert call(lib, **kw, ws_bytes=need - 1) == WS
                assert call(lib, **{**kw, "ws": 0}, ws_bytes=0) == WS
    for bad in ((0, 64, 1, 128, 128), (1, -1, 1, 128, 128), (1, 64, 0, 128, 128), (1, 64, 1, 96, 128),
                (1, 64, 1, 128, 32)):
        assert K.kda_linear_chunk_workspace_size(*bad) == 0
    assert lib.kda_linear_chunk_workspace_size(1, 64, 1, 128, 128, 9, 0) == 0


def test_forward_refusals(lib):
    assert fwd(lib, o=0) == INV
    assert fwd(lib, o_dt=3) == INV
    assert fwd(lib, o=Q + 64) == INV                       # o overlaps q
    assert fwd(lib, o=G) == INV
    assert fwd(lib, h0=H0, o=H0) == INV
    assert fwd(lib, hT=V) == INV                           # final state overlaps v
    assert fwd(lib, hT=O) == INV
    assert fwd(lib, h0=H0, hT=H0 + 4096) == INV            # partial overlap
    assert fwd(lib, o=O + 8) == UNS
    assert fwd(lib, hT=HT + 4) == UNS


def test_backward_refusals(lib):
    outs = dict(dq=DQ, dk_=DK, dv_=DV, dh0=DH)
    for name in ("do", "dq", "dk_", "dv_"):
        assert bwd(lib, **{name: 0}) == INV, name
        assert bwd(lib, **{name: FAKE + 0xF0000008}) == UNS, name
    for name in outs:
        for other in (Q, KK, V, DO, G, WSP):
            assert bwd(lib, **{name: other}) == INV, (name, other)
        assert bwd(lib, h0=H0, **{name: H0}) == INV
        assert bwd(lib, dhT=HT, **{name: HT}) == INV
        for other in outs:
            if other != name:
                assert bwd(lib, **{**outs, name: outs[other]}) == INV, (name, other)


def test_decode_refusals(lib):
    d = lambda **kw: lib.kda_linear_decode_step(                                   # noqa: E731
        P(kw.get("q", Q)), P(KK), P(V), kw.get("dt", 1), P(kw.get("g", G)), P(kw.get("S", HT)),
        P(kw.get("o", O)), kw.get("odt", 1), kw.get("N", 4), kw.get("H", 2), kw.get("dk", 128), 128,
        kw.get("scale", 1.0), None)
    for bad in (dict(dt=5), dict(odt=9), dict(N=-1), dict(H=0), dict(q=0), dict(g=0), dict(S=0), dict(o=0),
                dict(o=HT + 64), dict(S=Q), dict(o=KK), dict(S=G), dict(scale=float("nan"))):
        assert d(**bad) == INV, bad
    for bad in (dict(dk=32), dict(q=Q + 4), dict(S=HT + 8), dict(o=O + 2), dict(g=G + 1),
                dict(N=1 << 23, H=4)):
        assert d(**bad) == UNS, bad
    assert d(N=0, q=0, S=0, o=0) == 0                      # nothing to do


def test_state_cache_refusals(lib):
    def store(st=H0, sl=CU, c=Q, code=0, sc=G, N=4, n=8, H=2, dk=128, dv=128, group=64):
        return lib.kda_state_store(P(st), P(sl), P(c), code, P(sc), N, n, H, dk, dv, group, None)

    def load(st=H0, sl=CU, c=Q, code=0, sc=G, N=4, n=8, H=2, dk=128, dv=128, group=64):
        return lib.kda_state_load(P(c), code, P(sc), P(sl), P(st), N, n, H, dk, dv, group, None)

    for call in (store, load):
        for bad in (dict(code=2), dict(code=-1), dict(N=-1), dict(n=0), dict(H=0), dict(group=0),
                    dict(st=0), dict(c=0), dict(sc=0), dict(sl=0, N=9), dict(st=Q), dict(st=G)):
            assert call(**bad) == INV, bad
        for bad in (dict(dk=96), dict(dv=256), dict(group=16), dict(group=96), dict(group=128, dv=64),
                    dict(st=H0 + 4), dict(c=Q + 4), dict(sc=G + 2), dict(sl=CU + 2),
                    dict(N=1 << 30, n=1 << 30, H=64)):
            assert call(**bad) == UNS, bad
        assert call(N=0, st=0, c=0, sc=0) == 0             # nothing to do
    assert store(c=G) == INV and store(c=CU) == INV and store(sc=CU) == INV


# ------------------------------------------------------------------------------------ the binding

B, T, H, D = 1, 8, 2, 64


def args(**over):
    d = dict(q=torch.zeros(B, T, H, D, dtype=bf), k=torch.zeros(B, T, H, D, dtype=bf),
             v=torch.zeros(B, T, H, D, dtype=bf), g=torch.zeros(H))
    d.update(over)
    return d


def test_binding_host_tensors():
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kda_linear_chunk_fwd(**args())
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kda_linear_chunk_bwd(**args(), do=torch.zeros(B, T, H, D, dtype=bf))
    one = {n: x[0] if x.dim() == 4 else x for n, x in args().items()}
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kda_linear_decode_step(**one, state=torch.zeros(T, H, D, D))
    codes, scales = torch.zeros(2, H, D, D, dtype=torch.int8), torch.zeros(2, H, D, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kda_state_store(torch.zeros(2, H, D, D), codes, scales)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kda_state_load(codes, scales)


@pytest.mark.parametrize("over, what", [
    (dict(k=torch.zeros(B, T, H, D + 1, dtype=bf)), "k must have shape"),
    (dict(k=torch.zeros(B, T, H, D)), "share one dtype"),
    (dict(v=torch.zeros(B, T + 1, H, D, dtype=bf)), "v must have shape"),
    (dict(v=torch.zeros(B, T, H, dtype=bf)), "v must be a"),
    (dict(q=torch.zeros(T, H, D, dtype=bf)), "q must be a"),
    (dict(q=torch.zeros(B, T, H, D, dtype=torch.float16)), "q must be one of"),
    (dict(g=torch.zeros(H + 1)), "g must have shape"),
    (dict(g=torch.zeros(H, dtype=bf)), "g must be one of"),
    (dict(q=torch.zeros(B, T, H, 2 * D, dtype=bf)[..., ::2]), "contiguous"),
    (dict(initial_state=torch.zeros(2, H, D, D)), "initial_state must have shape"),
    (dict(initial_state=torch.zeros(B, H, D, D, dtype=bf)), "initial_state must be one of"),
    (dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int64)), "cu_seqlens must be one of"),
    (dict(cu_seqlens=torch.tensor([0], dtype=torch.int32)), "at least two"),
])
def test_binding_prefill_arguments(over, what):
    with pytest.raises(ValueError, match=what):
        K.kda_linear_chunk_fwd(**args(**over))
    with pytest.raises(ValueError, match=what):
        K.kda_linear_chunk_bwd(**args(**over), do=torch.zeros(B, T, H, D, dtype=bf))


def test_binding_other_arguments():
    do = torch.zeros(B, T, H, D, dtype=bf)
    with pytest.raises(ValueError, match="needs B == 1"):
        K.kda_linear_chunk_fwd(*(torch.zeros(2, T, H, D, dtype=bf) for _ in range(3)), torch.zeros(H),
                               cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(ValueError, match="o must have shape"):
        K.kda_linear_chunk_fwd(**args(), o=torch.zeros(B, T, H, D + 1, dtype=bf))
    with pytest.raises(ValueError, match="do must be one of"):
        K.kda_linear_chunk_bwd(**args(), do=do.float())
    with pytest.raises(TypeError, match="do must be"):
        K.kda_linear_chunk_bwd(**args(), do=None)
    with pytest.raises(ValueError, match="dq must be one of"):
        K.kda_linear_chunk_bwd(**args(), do=do, dq=do.float())
    with pytest.raises(ValueError, match="d_final_state must have shape"):
        K.kda_linear_chunk_bwd(**args(), do=do, d_final_state=torch.zeros(B, H, D, D + 1))
    one = {n: x[0] if x.dim() == 4 else x for n, x in args().items()}
    with pytest.raises(ValueError, match="state must have shape"):
        K.kda_linear_decode_step(**one, state=torch.zeros(T, H, D, D + 1))
    with pytest.raises(ValueError, match="q must be a"):
        K.kda_linear_decode_step(**args(), state=torch.zeros(T, H, D, D))
    codes, scales = torch.zeros(2, H, D, D, dtype=torch.int8), torch.zeros(2, H, D, 1)
    st = torch.zeros(2, H, D, D)
    with pytest.raises(ValueError, match="codes must be one of"):
        K.kda_state_store(st, codes.view(torch.uint8), scales)
    with pytest.raises(ValueError, match="scales must have shape"):
        K.kda_state_store(st, codes, scales[:1])
    with pytest.raises(ValueError, match="must end in dv / group"):
        K.kda_state_store(st, codes, torch.zeros(2, H, D, 3))
    with pytest.raises(ValueError, match="states must have shape"):
        K.kda_state_store(st[:1], codes, scales, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="slots must be one of"):
        K.kda_state_load(codes, scales, torch.zeros(2, dtype=torch.int64))
