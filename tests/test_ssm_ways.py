"""The chunked form of ddt in ssm_ways against the token-by-token one in ssm_ref, and whether the bound that the GPU tests
take from it tells a right ddt from a wrong one."""
import pytest
import torch

import ssm_ref as R
import ssm_ways as W

BOUND = 2.0 ** -16               # of the magnitudes, as in test_gpu_ssm_ddt


def batch(lens, H=3, G=1, dk=64, dv=64, state=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).double()                     # noqa: E731
    T, N = sum(lens), len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d = dict(x=r(1, T, H, dv), dt=2 * r(1, T, H), A=-(0.5 + 8 * torch.rand(H, generator=g).double()), B=r(1, T, G, dk),
             C=r(1, T, G, dk), dy=r(1, T, H, dv), bias=-2 + r(H), cu=cu)
    if state:
        d.update(h0=r(N, H, dk, dv), dhT=r(N, H, dk, dv))
    return d


@pytest.mark.parametrize("chunk", [1, 32, 64])
@pytest.mark.parametrize("lens,G", [([1], 1), ([70], 3), ([64, 0, 33, 130], 1)])
def test_equal_forms(chunk, lens, G):
    d = batch(lens, G=G, dk=8, dv=12)
    ref = R.scan_grads(**d)["ddt"]
    got = W.ddt(**d, chunk=chunk)
    assert (got - ref).abs().max() <= 1e-12 * W.ddt(**d, chunk=chunk, magnitude=True).max()


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("chunk", [32, 64])
def test_the_bound_tells(chunk, seed):
    """1290 tokens: the bound lies below a quarter of most entries, and a wrong ddt lies beyond it nearly everywhere."""
    d = batch([1290], seed=seed)
    ref = W.ddt(**d, chunk=chunk)
    bound = BOUND * W.ddt(**d, chunk=chunk, magnitude=True)
    share = lambda t: t.double().mean().item()                               # noqa: E731
    assert share(bound < ref.abs() / 4) > 0.85
    borders = [*range(0, 1290, chunk), 1290]
    alone = {**d, "cu": borders, "h0": None, "dhT": None}                    # nothing goes from chunk to chunk
    beyond = lambda wrong: (wrong - ref).abs() > bound                       # noqa: E731
    for wrong in (ref.roll(1, 1), 0 * ref, W.ddt(**{**d, "bias": None})):
        assert share(beyond(wrong)) > 0.9
    assert share(beyond(W.ddt(**alone))[:, chunk:-1:chunk]) > 0.6            # the chunks' first tokens
