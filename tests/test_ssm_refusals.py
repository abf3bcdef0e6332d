"""Refusals of the convolution, scan and slot calls, in the C ABI and in the binding.  CPU only: the pointers are never
dereferenced, each call fails validation (or has nothing to do) before any device work."""
import ctypes

import pytest
import torch

from gated_delta_rule_60_amd import kda as K

FAKE = 1 << 40
INV, UNS, WS = 1, 2, 3
(X, DT, B_, C_, A, BIAS, D, H0, HT, CU, Y, WSP, DY, DX, DDT, DB, DC, DA, DD, DBI, DH0, DHT, S,
 SL) = (FAKE + i * 0x10000000 for i in range(24))
bf, f32 = torch.bfloat16, torch.float32
nan = float("nan")


def P(x):
    return ctypes.c_void_p(x) if x else None


@pytest.fixture(scope="module")
def lib():
    return K.load_library()


def conv_fwd(lib, x=X, ldx=64, dt=1, w=B_, b=BIAS, h0=0, hT=0, cu=0, y=Y, ldy=64, B=1, T=100, N=1, C=64, W=4):
    return lib.kda_conv_fwd(P(x), ldx, dt, P(w), P(b), P(h0), P(hT), P(cu), P(y), ldy, B, T, N, C, W, 1, None)


def conv_bwd(lib, x=X, ldx=64, dt=1, w=B_, b=BIAS, h0=0, cu=0, dy=DY, lddy=64, dhT=0, dx=DX, lddx=64, dw=DA, db=DBI,
             dh0=0, B=1, T=100, N=1, C=64, W=4, ws=WSP, ws_bytes=1 << 24):
    return lib.kda_conv_bwd(P(x), ldx, dt, P(w), P(b), P(h0), P(cu), P(dy), lddy, P(dhT), P(dx), lddx, P(dw), P(db),
                            P(dh0), B, T, N, C, W, 1, P(ws), ws_bytes, None)


def conv_step(lib, x=X, ldx=64, dt=1, w=B_, b=BIAS, win=S, slots=SL, y=Y, ldy=64, N=3, n_slots=8, C=64, W=4):
    return lib.kda_conv_step(P(x), ldx, dt, P(w), P(b), P(win), P(slots), P(y), ldy, N, n_slots, C, W, 1, None)


def fwd(lib, x=X, ldx=256, dt=DT, lddt=4, B=B_, ldb=128, C=C_, ldc=128, in_dt=1, A_=A, bias=BIAS, D_=D, h0=0, hT=0,
        cu=0, y=Y, ldy=256, y_dt=1, nb=1, T=100, N=1, H=4, G=2, dk=64, dv=64, ws=WSP, ws_bytes=1 << 27):
    return lib.kda_ssm_chunk_fwd(P(x), ldx, P(dt), lddt, P(B), ldb, P(C), ldc, in_dt, P(A_), P(bias), P(D_), P(h0), P(hT),
                                 P(cu), P(y), ldy, y_dt, nb, T, N, H, G, dk, dv, P(ws), ws_bytes, None)


def bwd(lib, x=X, ldx=256, dt=DT, lddt=4, B=B_, ldb=128, C=C_, ldc=128, in_dt=1, A_=A, bias=BIAS, D_=D, h0=0, cu=0,
        dy=DY, lddy=256, dhT=0, dx=DX, lddx=256, ddt=DDT, ldddt=4, dB=DB, lddb=128, dC=DC, lddc=128, dA=DA, dD=DD,
        dbias=DBI, dh0=0, nb=1, T=100, N=1, H=4, G=2, dk=64, dv=64, ws=WSP, ws_bytes=1 << 27):
    return lib.kda_ssm_chunk_bwd(P(x), ldx, P(dt), lddt, P(B), ldb, P(C), ldc, in_dt, P(A_), P(bias), P(D_), P(h0), P(cu),
                                 P(dy), lddy, P(dhT), P(dx), lddx, P(ddt), ldddt, P(dB), lddb, P(dC), lddc, P(dA), P(dD),
                                 P(dbias), P(dh0), nb, T, N, H, G, dk, dv, P(ws), ws_bytes, None)


def step(lib, x=X, ldx=256, dt=DT, lddt=4, B=B_, ldb=128, C=C_, ldc=128, in_dt=1, A_=A, bias=BIAS, D_=D, state=S,
         slots=SL, y=Y, ldy=256, y_dt=1, N=3, n_slots=8, H=4, G=2, dk=64, dv=64):
    return lib.kda_ssm_decode_step(P(x), ldx, P(dt), lddt, P(B), ldb, P(C), ldc, in_dt, P(A_), P(bias), P(D_), P(state),
                                   P(slots), P(y), ldy, y_dt, N, n_slots, H, G, dk, dv, None)


def each(call, lib, want, cases):
    for bad in cases:
        assert call(lib, **bad) == want, (call.__name__, bad)


@pytest.mark.parametrize("call", [conv_fwd, conv_bwd])
def test_conv(lib, call):
    each(call, lib, INV, [dict(dt=2), dict(B=0), dict(T=-1), dict(N=2), dict(B=2, N=2, cu=CU), dict(C=0), dict(W=0),
                          dict(x=0), dict(w=0), dict(ldx=63)])
    each(call, lib, UNS, [dict(W=1), dict(W=5), dict(x=X + 1), dict(w=B_ + 2), dict(cu=CU + 2, N=1), dict(ldx=1 << 24),
                          dict(T=1 << 32), dict(N=1 << 25, B=1 << 25, T=0), dict(C=1 << 24, ldx=1 << 24)])


def test_conv_outputs(lib):
    each(conv_fwd, lib, INV, [dict(y=0), dict(ldy=10), dict(y=X), dict(y=X + 64), dict(hT=H0, h0=H0), dict(hT=H0 + 2, h0=H0),
                              dict(y=B_), dict(hT=Y), dict(cu=CU, y=CU), dict(y=X + 128 * 50, ldy=128)])
    each(conv_bwd, lib, INV, [dict(dy=0), dict(dx=0), dict(dw=0), dict(dx=X), dict(dx=DY), dict(dw=B_), dict(db=DA),
                              dict(dh0=H0, h0=H0), dict(dh0=DHT, dhT=DHT), dict(ws=X), dict(ws=DX), dict(lddy=3),
                              dict(lddx=3)])
    each(conv_bwd, lib, WS, [dict(ws=0), dict(ws_bytes=0), dict(ws_bytes=K.kda_conv_bwd_workspace_size(1, 100, 64, 4) - 1)])
    each(conv_bwd, lib, UNS, [dict(ws=WSP + 4), dict(dw=DA + 1), dict(dx=DX + 1)])
    for bad in ((0, 1, 1, 4), (1, -1, 1, 4), (1, 1, 0, 4), (1, 1, 1, 1), (1, 1, 1, 5)):
        assert K.kda_conv_bwd_workspace_size(*bad) == 0


def test_conv_step(lib):
    each(conv_step, lib, INV, [dict(dt=5), dict(N=-1), dict(n_slots=0), dict(C=0), dict(slots=0, N=9), dict(x=0), dict(win=0),
                               dict(y=0), dict(w=0), dict(y=X), dict(y=S), dict(win=X), dict(slots=S), dict(ldx=1), dict(ldy=1)])
    each(conv_step, lib, UNS, [dict(W=5), dict(W=1), dict(slots=SL + 1), dict(win=S + 1), dict(N=1 << 24, n_slots=1 << 24)])
    assert conv_step(lib, N=0, x=0, y=0) == 0


@pytest.mark.parametrize("call", [fwd, bwd])
def test_scan(lib, call):
    each(call, lib, INV, [dict(in_dt=3), dict(nb=0), dict(T=-1), dict(N=2), dict(nb=2, N=2, cu=CU), dict(H=0), dict(G=0),
                          dict(G=3), dict(x=0), dict(dt=0), dict(B=0), dict(C=0), dict(A_=0), dict(ldx=255), dict(lddt=3),
                          dict(ldb=127), dict(ldc=100), dict(ws=X), dict(ws=A), dict(h0=H0, ws=H0), dict(A_=0, T=0)])
    each(call, lib, UNS, [dict(dk=96), dict(dv=32), dict(x=X + 8), dict(B=B_ + 2), dict(C=C_ + 4), dict(dt=DT + 1),
                          dict(A_=A + 2), dict(ldx=260), dict(ldb=129), dict(ldc=132), dict(ldx=1 << 24), dict(h0=H0 + 4),
                          dict(ws=WSP + 8), dict(cu=CU + 2), dict(H=65536, G=1, ldx=1 << 22, lddt=65536, T=0),
                          dict(N=1 << 21, nb=1 << 21, T=0), dict(T=1 << 31)])


def test_scan_outputs(lib):
    each(fwd, lib, INV, [dict(y=0), dict(y_dt=9), dict(ldy=255), dict(y=X), dict(y=DT), dict(hT=H0 + 16, h0=H0), dict(hT=Y),
                         dict(y=H0, h0=H0), dict(hT=WSP)])
    each(fwd, lib, UNS, [dict(y=Y + 8), dict(ldy=258), dict(hT=HT + 4)])
    need = K.kda_ssm_chunk_workspace_size(1, 4096, 4, 2, 64, 64)
    assert need > 0
    far = dict(T=4096, x=FAKE, y=FAKE + (1 << 34), B=FAKE + (2 << 34), C=FAKE + (3 << 34), ws=FAKE + (4 << 34))
    each(fwd, lib, WS, [dict(far, ws_bytes=need - 1), dict(far, ws=0)])
    each(bwd, lib, INV, [dict(dy=0), dict(dx=0), dict(ddt=0), dict(dB=0), dict(dC=0), dict(dA=0), dict(dx=X), dict(dB=DC),
                         dict(dx=DY), dict(dA=DD), dict(dbias=A), dict(dh0=H0, h0=H0), dict(dh0=DHT, dhT=DHT), dict(lddx=1),
                         dict(ldddt=1), dict(lddb=1), dict(lddc=1), dict(lddy=1)])
    each(bwd, lib, UNS, [dict(dx=DX + 8), dict(dB=DB + 8), dict(ddt=DDT + 1), dict(dA=DA + 2), dict(lddx=257), dict(dh0=DH0 + 4)])
    each(bwd, lib, WS, [dict(ws=0), dict(ws_bytes=K.kda_ssm_chunk_workspace_size(1, 100, 4, 2, 64, 64, backward=True) - 1)])
    for bad in ((0, 1, 1, 1, 64, 64), (1, -1, 1, 1, 64, 64), (1, 1, 0, 1, 64, 64), (1, 1, 4, 3, 64, 64), (1, 1, 4, 2, 32, 64),
                (1, 1, 4, 2, 64, 65), (1, 1 << 40, 4, 2, 64, 64)):
        assert K.kda_ssm_chunk_workspace_size(*bad) == 0


def test_chunks_of_the_gradients(lib):
    """Sizes that the forward call takes but the gradients' grids would not hold."""
    size = lambda T, H, dtype, backward: K.kda_ssm_chunk_workspace_size(1, T, H, H, 64, 64, dtype, backward)
    T = 128 * ((1 << 21) - 64)
    assert size(T, 1, f32, False) > 0 and size(T, 1, f32, True) == 0
    assert size(T // 2, 1, f32, True) > 0 and size(T, 1, bf, True) > 0
    far = dict(H=1, G=1, in_dt=0, T=T, **{k: (i + 1) << 44 for i, k in enumerate(("x", "dt", "B", "C", "dy", "dx", "ddt", "dB", "dC"))})
    assert bwd(lib, **far, ws_bytes=0) == UNS
    assert bwd(lib, **{**far, "T": T // 2}, ws_bytes=0) == WS


def test_side_by_side_rows(lib):
    """Gradients in one wider row are disjoint where their columns are, and only there.  (A call that passes the checks
    would launch: so one more argument is wrong in a way that is found later.)"""
    ld, es = 512, 2
    side = dict(lddx=ld, lddb=ld, lddc=ld, dx=DX, dB=DX + 256 * es, dC=DX + 384 * es)
    assert bwd(lib, **side, ws_bytes=0) == WS
    for shift in ("dB", "dC"):
        assert bwd(lib, **{**side, shift: side[shift] - 16}) == INV
    assert bwd(lib, **{**side, "dC": side["dC"] + 16}) == INV          # runs into the next row's dx


def test_scan_step(lib):
    each(step, lib, INV, [dict(in_dt=2), dict(y_dt=2), dict(N=-1), dict(n_slots=0), dict(H=0), dict(G=3), dict(slots=0, N=9),
                          dict(x=0), dict(dt=0), dict(B=0), dict(C=0), dict(A_=0), dict(state=0), dict(y=0), dict(y=X), dict(y=S),
                          dict(state=X), dict(slots=S), dict(ldx=1), dict(ldy=1)])
    each(step, lib, UNS, [dict(dk=32), dict(dv=256), dict(x=X + 8), dict(state=S + 8), dict(slots=SL + 1), dict(ldb=132 + 1),
                          dict(N=1 << 22, n_slots=1 << 22)])
    assert step(lib, N=0, x=0, y=0) == 0


def arrays(*planes):
    return (ctypes.c_void_p * len(planes))(*planes)


def sizes(*n):
    return (ctypes.c_int64 * len(n))(*n)


def test_slots(lib):
    def fork(planes=arrays(S), b=sizes(256), n=1, refs=A, parents=SL, children=Y, N=2, n_slots=8, ws=WSP, ws_bytes=1 << 20):
        return lib.kda_slots_fork(planes, b, n, P(refs), P(parents), P(children), N, n_slots, P(ws), ws_bytes, None)

    def compact(planes=arrays(S), b=sizes(256), n=1, refs=A, table=SL, n_table=4, used=Y, n_slots=8, ws=WSP, ws_bytes=1 << 20):
        return lib.kda_slots_compact(planes, b, n, P(refs), P(table), n_table, P(used), n_slots, P(ws), ws_bytes, None)

    def copy(src=arrays(X), dst=arrays(S), b=sizes(256), n=1, a=SL, c=Y, N=2, n_src=8, n_dst=8):
        return lib.kda_slots_copy(src, dst, b, n, P(a), P(c), N, n_src, n_dst, None)

    for call in (fork, compact):
        for bad in (dict(n_slots=0), dict(n=0), dict(planes=None), dict(b=None), dict(planes=arrays(0)), dict(b=sizes(0)),
                    dict(refs=0), dict(refs=S + 16), dict(ws=S), dict(planes=arrays(S, S + 16), b=sizes(256, 256), n=2)):
            assert call(**bad) == INV, bad
        for bad in (dict(n_slots=(1 << 20) + 1), dict(planes=arrays(S + 8)), dict(planes=arrays(*[S] * 5), b=sizes(*[256] * 5), n=5),
                    dict(refs=A + 1), dict(ws=WSP + 4), dict(b=sizes(1 << 41))):
            assert call(**bad) == UNS, bad
        for bad in (dict(ws=0), dict(ws_bytes=8)):
            assert call(**bad) == WS, bad
    assert fork(N=-1) == INV and fork(children=0) == INV and fork(children=SL) == INV and fork(N=0) == 0
    assert compact(n_table=-1) == INV and compact(table=0) == INV and compact(used=0) == INV and compact(used=SL) == INV
    for bad in (dict(N=-1), dict(n_src=0), dict(n_dst=0), dict(a=0, N=9), dict(c=0, N=9), dict(dst=arrays(X)), dict(dst=arrays(X + 16)),
                dict(a=S), dict(c=S + 16), dict(n=0), dict(src=None)):
        assert copy(**bad) == INV, bad
    for bad in (dict(a=SL + 1), dict(src=arrays(X + 4)), dict(b=sizes(1 << 40), N=1, a=SL)):
        assert copy(**bad) == UNS, bad
    assert copy(N=0) == 0
    for fn in (lib.kda_slots_retain, lib.kda_slots_release):
        assert fn(P(A), P(SL), -1, 8, None) == INV and fn(P(A), P(SL), 1, 0, None) == INV
        assert fn(None, P(SL), 1, 8, None) == INV and fn(P(A), None, 1, 8, None) == INV
        assert fn(P(A), P(A + 4), 2, 8, None) == INV
        assert fn(P(A + 1), P(SL), 1, 8, None) == UNS and fn(P(A), P(SL), 1, (1 << 20) + 1, None) == UNS
        assert fn(None, None, 0, 8, None) == 0
    assert K.kda_slots_workspace_size(0) == 0 and K.kda_slots_workspace_size(8, -1) == 0


def test_binding(lib):
    """Wrong shapes, types, strides and devices raise before the library is called (CPU tensors are refused last)."""
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    for bad in (lambda: K.kda_conv_fwd(x[0], w), lambda: K.kda_conv_fwd(x, w[:4]), lambda: K.kda_conv_fwd(x, w.to(bf)),
                lambda: K.kda_conv_fwd(x, w, torch.zeros(7)), lambda: K.kda_conv_fwd(x, w, initial_state=torch.zeros(2, 4, 8)),
                lambda: K.kda_conv_fwd(x.transpose(0, 1), w), lambda: K.kda_conv_fwd(x.half(), w), lambda: K.kda_conv_fwd(x, w),
                lambda: K.kda_conv_fwd(x[:, :, ::2], w[:4]), lambda: K.kda_conv_fwd(x, w, cu_seqlens=torch.zeros(3, dtype=torch.int32)),
                lambda: K.kda_conv_fwd(x[:1].expand(2, 5, 8), w), lambda: K.kda_conv_bwd(x, w, x.to(bf)),
                lambda: K.kda_conv_step(x, w, x), lambda: K.kda_conv_step(x[0], w, torch.zeros(4, 2, 8))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    xs, dt, A_ = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 4), torch.zeros(4)
    Bm = torch.zeros(2, 5, 2, 64)
    f = K.kda_ssm_chunk_fwd
    for bad in (lambda: f(xs, dt, A_, Bm, Bm), lambda: f(xs, dt, A_, Bm[:, :, :1].expand(2, 5, 3, 64), Bm), lambda: f(xs, dt[:, :4], A_, Bm, Bm),
                lambda: f(xs, dt.to(bf), A_, Bm, Bm), lambda: f(xs, dt, A_.double(), Bm, Bm), lambda: f(xs, dt, A_, Bm, Bm, D=torch.zeros(3)),
                lambda: f(xs, dt, A_, Bm, Bm, initial_state=torch.zeros(1, 4, 64, 64)), lambda: f(xs, dt, A_, Bm, Bm, y=xs[:1]),
                lambda: f(xs, dt, A_, Bm, Bm, cu_seqlens=torch.zeros(2, dtype=torch.int32)),
                lambda: K.kda_ssm_chunk_bwd(xs, dt, A_, Bm, Bm, xs[:1]), lambda: K.kda_ssm_chunk_bwd(xs, dt, A_, Bm, Bm, None),
                lambda: K.kda_ssm_decode_step(xs[0], dt[0], A_, Bm[0], Bm[0], torch.zeros(5, 4, 64, 32)),
                lambda: K.kda_ssm_decode_step(xs[0], dt[0], A_, Bm[0], Bm[0], torch.zeros(5, 4, 64, 64), slots=torch.zeros(5))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    pool, refs = torch.zeros(6, 3), torch.zeros(6, dtype=torch.int32)
    for bad in (lambda: K.kda_slots_fork([], refs, 1), lambda: K.kda_slots_fork(pool, refs[:5], 1), lambda: K.kda_slots_fork(pool, refs, 1.5),
                lambda: K.kda_slots_fork([pool, pool[:5]], refs, 1), lambda: K.kda_slots_fork(pool.t(), refs, 1),
                lambda: K.kda_slots_fork(pool[:, :0], refs, 1), lambda: K.kda_slots_fork(pool, refs, refs.long()),
                lambda: K.kda_slots_compact(pool, refs, table=refs.long()), lambda: K.kda_slots_compact(pool, refs),
                lambda: K.kda_slots_copy(pool, torch.zeros(4, 2)), lambda: K.kda_slots_copy(pool, pool.clone(), refs, refs[:2]),
                lambda: K.kda_slots_release(refs.long(), refs), lambda: K.kda_slots_release(refs, refs)):
        with pytest.raises((ValueError, TypeError)):
            bad()
