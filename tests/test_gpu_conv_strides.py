"""The convolution at the largest stride it takes, 2^24 bytes from token to token: offsets inside a run of 128 tokens and
its neighbours pass 2^31.  The same inputs row after row give the same bits."""
import pytest
import torch

from gated_delta_rule_60_amd import kda as K
from kda_testutil import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,C", [(torch.bfloat16, 64), (torch.bfloat16, 7), (torch.float32, 12)])
def test_largest_stride(dtype, C):
    T, row = 140, (1 << 24) // dtype.itemsize
    wide = torch.empty((1, T, row), dtype=dtype, device=DEV)
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(1, T, C, generator=g).to(dtype).to(DEV) for _ in range(2))
    w, b = torch.randn(C, 4, generator=g).to(DEV), torch.randn(C, generator=g).to(DEV)
    at = lambda i: wide[..., row - 64 * (4 - i):row - 64 * (4 - i) + C]             # noqa: E731  (the rows' last columns)
    at(0).copy_(x)
    at(1).copy_(dy)
    for cu in (None, torch.tensor([0, 5, 140], dtype=torch.int32, device=DEV)):
        y, _ = K.kda_conv_fwd(x, w, b, cu_seqlens=cu)
        want = K.kda_conv_bwd(x, w, dy, b, cu_seqlens=cu)
        K.kda_conv_fwd(at(0), w, b, cu_seqlens=cu, y=at(2))
        got = K.kda_conv_bwd(at(0), w, at(1), b, cu_seqlens=cu, dx=at(3))
        torch.cuda.synchronize()
        assert torch.equal(at(2), y) and torch.equal(at(3), want[0])
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert torch.equal(at(0), x) and torch.equal(at(1), dy)
