"""How the scan's and the convolution's calls may be made: blocks of heads of every kind, workspaces with anything in
them, two streams at once, rows beyond 4 GB, the debug check.  Results are compared with the fp64 reference at the
tolerances of test_gpu_ssm, or bit for bit with the same call made another way (sums have a fixed order)."""
import pytest
import torch

import ssm_ref as R
from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV
from test_gpu_ssm import backward, bf, check_backward, check_forward, f32, forward, make

pytestmark = pytest.mark.gpu


def same(a, b):
    for s, t in zip(a, b):
        assert (s is None) == (t is None) and (s is None or torch.equal(s, t))


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("n_seqs,hg", [(300, (3, 1)), (140, (3, 1)), (130, (10, 2)), (70, (5, 1))])
def test_blocks_of_heads(dtype, dk, dv, n_seqs, hg):
    """Many short sequences: all of a group's heads in one workgroup of the gradients (300 x 3, 130 x 5 of 2 groups), or in
    two (140 x 3: two heads and one; 70 x 5: two, two and one)."""
    lens = [n * 7 % 5 for n in range(n_seqs)]
    d = make(dtype, lens, *hg, dk, dv, packed=True, state=True, seed=5)
    check_forward(d, dtype)
    check_backward(d, dtype)


def test_one_head_more_than_a_block_over_chunks():
    """Sequences of several chunks, heads of a workgroup one after the other: 130 chunks, blocks of two heads and one."""
    d = make(bf, [8320], 3, 1, 128, 64, packed=False, state=False, seed=6)
    check_backward(d, bf)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("lens", [[1500], [40, 0, 1300, 7]])
def test_any_workspace(dtype, lens):
    """A workspace full of NaNs gives the bits of one full of zeros."""
    d = make(dtype, lens, 4, 2, 128, 64, packed=len(lens) > 1, state=True, seed=7)
    got = []
    for fill in (0, 255):
        size = lambda back: K.kda_ssm_chunk_workspace_size(len(lens), sum(lens), 4, 2, 128, 64, dtype, back)   # noqa: E731
        ws = [torch.full((max(16, size(back)),), fill, dtype=torch.uint8, device=DEV) for back in (False, True)]
        got.append([*forward(d, workspace=ws[0]), *backward(d, workspace=ws[1])])
    torch.cuda.synchronize()
    same(*got)


def test_two_streams_at_once():
    """Two batches on two streams, call by call in turn, each as if it were alone."""
    ds = [make(bf, [1100], 4, 1, 128, 64, packed=False, state=True, seed=s) for s in (8, 9)]
    want = [[*forward(d), *backward(d)] for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for call in (forward, backward):
        for i, (s, d) in enumerate(zip(streams, ds)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] += call(d)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        same(w, g)


def test_rows_beyond_4_gb():
    """Rows 64 KB apart: the last tokens' offsets do not fit 32 bits.  The same inputs row after row give the same bits."""
    T, row = 70000, 32768
    wide = torch.empty((1, T, row), dtype=bf, device=DEV)
    g = torch.Generator().manual_seed(10)
    near = torch.randn(1, T, 64 + 2 * 64 + 16, generator=g).to(bf).to(DEV)
    cols = near.shape[-1]
    wide[..., :cols].copy_(near)
    parts = lambda t: (t[..., :64].unflatten(-1, (1, 64)), t[..., 64:128].unflatten(-1, (1, 64)),   # noqa: E731
                       t[..., 128:192].unflatten(-1, (1, 64)), t[..., 192:193])
    A = torch.tensor([-2.0], device=DEV)
    w = torch.randn(64, 4, generator=g).to(DEV)
    got = []
    for t in (near, wide):
        x, B, C, dt = parts(t)
        y, hT = K.kda_ssm_chunk_fwd(x, dt, A, B, C)
        u, _ = K.kda_conv_fwd(t[..., :64], w)
        du = K.kda_conv_bwd(t[..., :64], w, t[..., 64:128])
        got.append([y, hT, u, *[z for z in du if z is not None], *K.kda_ssm_chunk_bwd(x, dt, A, B, C, x)[:5]])
    torch.cuda.synchronize()
    same(*got)
    # and outputs into such rows
    x, B, C, dt = parts(near)
    out = wide[..., 1024:1024 + 64].unflatten(-1, (1, 64))
    K.kda_ssm_chunk_fwd(x, dt, A, B, C, y=out)
    K.kda_conv_fwd(near[..., :64], w, y=wide[..., 2048:2048 + 64])
    torch.cuda.synchronize()
    assert torch.equal(out, got[0][0]) and torch.equal(wide[..., 2048:2048 + 64], got[0][2])
    assert torch.equal(wide[..., :cols], near)


def test_debug_check(monkeypatch):
    """KDA_DEBUG_VALIDATE refuses positive or NaN A and malformed offsets, and takes what is right."""
    d = make(bf, [30, 70], 2, 1, 64, 64, packed=True, state=True, seed=11)
    state = torch.zeros((1, 2, 64, 64), device=DEV)
    one = [d[k][0, :1].contiguous() for k in ("x", "dt", "B", "C")]
    x, dt, B, C = one
    conv = d["row"][..., :64].contiguous().to(DEV)
    w = torch.randn(64, 4).to(DEV)
    monkeypatch.setenv("KDA_DEBUG_VALIDATE", "1")
    forward(d)
    backward(d)
    K.kda_conv_fwd(conv, w, cu_seqlens=d["cu"])
    K.kda_ssm_decode_step(x, dt, d["A"], B, C, state)
    for bad in (0.5, float("nan")):
        e = dict(d, A=torch.tensor([-1.0, bad], device=DEV))
        for call in (lambda: forward(e), lambda: backward(e), lambda: K.kda_ssm_decode_step(x, dt, e["A"], B, C, state)):
            with pytest.raises(K.KDAError) as err:
                call()
            assert err.value.status == 1
    for cu in ([0, 80, 60], [1, 70, 100], [0, 70, 99]):
        e = dict(d, cu=torch.tensor(cu, dtype=torch.int32, device=DEV))
        for call in (lambda: forward(e), lambda: backward(e), lambda: K.kda_conv_fwd(conv, w, cu_seqlens=e["cu"]),
                     lambda: K.kda_conv_bwd(conv, w, conv, cu_seqlens=e["cu"])):
            with pytest.raises(K.KDAError) as err:
                call()
            assert err.value.status == 1


@pytest.mark.parametrize("dtype", [bf, f32])
def test_gradients_against_differences(dtype):
    """The gradients as slopes of the forward call itself: along a direction u, the change of <y, dy> + <hT, dhT>."""
    d = make(f32, [150], 2, 1, 64, 64, packed=False, state=True, seed=12, wide=False)
    if dtype is bf:                                  # (values of 16 bits; the calls run in fp32, whose differences show)
        for k in ("x", "B", "C", "dt", "dy"):
            d[k] = d[k].to(bf).float()
    names = ("x", "dt", "A", "B", "C", "D", "bias", "h0")
    got = dict(zip(names, backward(d)))
    g = torch.Generator().manual_seed(13)
    ref = lambda e: R.scan(*[R.f64(e[k].cpu()) for k in ("x", "dt", "A", "B", "C")], D=R.f64(e["D"].cpu()),   # noqa: E731
                           bias=R.f64(e["bias"].cpu()), h0=R.f64(e["h0"].cpu()))
    dy, dhT = R.f64(d["dy"].cpu()), R.f64(d["dhT"].cpu())
    for k in names:
        u = torch.randn(d[k].shape, generator=g).double()
        step = 1e-6
        ends = []
        for sign in (1, -1):
            e = {n: (d[n].cpu().double() if n in names else d[n]) for n in (*names, "dy", "dhT")}
            e[k] = e[k] + sign * step * u
            y, hT = ref(e)
            ends.append((y * dy).sum() + (hT * dhT).sum())
        slope = ((ends[0] - ends[1]) / (2 * step)).item()
        have = (got[k].double().cpu() * u).sum().item()
        terms = (got[k].double().cpu() * u).abs().sum().item()
        # the difference's own error is of the order step^2 of a third derivative, far below the terms' 2^-15
        assert abs(have - slope) <= 2.0 ** -15 * terms, (k, have, slope, terms)
