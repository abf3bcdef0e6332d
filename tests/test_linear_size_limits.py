"""The size limits include/kda.h states for the linear-attention and state-cache calls: one past each is
refused before any device work (CPU; the pointers are never dereferenced)."""
import pytest

from gated_delta_rule_60_amd import kda as K
from test_linear_refusals import CU, G, H0, HT, KK, O, P, Q, UNS, V, bwd, fwd


@pytest.fixture(scope="module")
def lib():
    return K.load_library()


@pytest.mark.parametrize("call", [fwd, bwd])
def test_prefill_and_gradients(lib, call):
    assert call(lib, H=32769, T=0) == UNS
    for N, H in (((1 << 21) + 1, 1), (1 << 20, 3), (65, 32768)):
        assert call(lib, B=N, N=N, H=H, T=0) == UNS
        assert call(lib, B=1, N=N, H=H, T=0, cu=CU) == UNS


def test_decode(lib):
    for N, H in ((1 << 24, 1), (1 << 12, 1 << 12), (1, 1 << 24)):
        assert lib.kda_linear_decode_step(P(Q), P(KK), P(V), 1, P(G), P(HT), P(O), 1, N, H, 64, 64, 1.0,
                                          None) == UNS


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 128)])
def test_state_cache(lib, dk, dv):
    for N, H in (((1 << 36) // (dk * dv), 1), ((1 << 36) // (dk * dv * 16), 16)):
        # a store of that many sequences needs as many slots only without a slot list
        assert lib.kda_state_store(P(H0), P(CU), P(Q), 0, P(G), N, 4, H, dk, dv, 64, None) == UNS
        assert lib.kda_state_load(P(Q), 0, P(G), P(CU), P(H0), N, 4, H, dk, dv, 64, None) == UNS
