"""One workspace, sized for the largest batch, for every smaller call of the scan and of the convolution's gradients:
the bits of a call with a workspace of its own."""
import pytest
import torch

from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV
from test_gpu_ssm import backward, bf, f32, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("H,G,dk,dv", [(4, 2, 64, 64), (2, 1, 128, 128)])
def test_one_workspace_for_all(dtype, H, G, dk, dv):
    most = lambda back: K.kda_ssm_chunk_workspace_size(40, 5000, H, G, dk, dv, dtype, back)   # noqa: E731
    ws = [torch.full((most(back),), 255, dtype=torch.uint8, device=DEV) for back in (False, True)]
    for lens, packed in (([5000], False), ([4097], False), ([4096], False), ([600] * 8, False), ([1, 3000, 0, 700], True),
                         ([64] * 40, True), ([9], False)):
        d = make(dtype, lens, H, G, dk, dv, packed=packed, state=True, seed=len(lens))
        want = [*forward(d), *backward(d)]
        got = [*forward(d, workspace=ws[0]), *backward(d, workspace=ws[1])]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b), lens


@pytest.mark.parametrize("dtype", [bf, f32])
def test_convolution(dtype):
    g = torch.Generator().manual_seed(1)
    ws = torch.empty(K.kda_conv_bwd_workspace_size(9, 2000, 96, 4), dtype=torch.uint8, device=DEV)
    for N, T, C, W in ((1, 2000, 96, 4), (9, 200, 96, 4), (9, 1, 96, 3), (2, 130, 7, 2)):
        x, dy = (torch.randn(N, T, C, generator=g).to(dtype).to(DEV) for _ in range(2))
        w = torch.randn(C, W, generator=g).to(DEV)
        want, got = K.kda_conv_bwd(x, w, dy), K.kda_conv_bwd(x, w, dy, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
