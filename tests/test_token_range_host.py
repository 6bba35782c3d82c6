"""CPU test of the temperatures that the token statistics' calls take."""
import os

import pytest

from response_replay_gb300 import binding as B

A = 1 << 20  # an aligned address that nothing reads: every call below is refused


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from response_replay_gb300 import build
        build.build()
    return B.lib()


@pytest.mark.parametrize("temp,want", [(0.0, B.LS_ERR_INVALID_ARG), (1e-7, B.LS_ERR_INVALID_ARG),
                                       (1e-6, B.LS_ERR_UNSUPPORTED), (9.9e-4, B.LS_ERR_UNSUPPORTED),
                                       (2e6, B.LS_ERR_INVALID_ARG)])
def test_backward_refuses_temperatures(lib, temp, want):
    for T in (0, 4):
        assert lib.ls_token_logp_bwd(A, B.LS_BF16, T, 100, 100, A, temp, A, A, 0, None, A, A, None, A + 65536, 100,
                                     None) == want


def test_lowest_temperature_of_the_backward(lib):
    # accepted, and without rows nothing is launched
    assert lib.ls_token_logp_bwd(A, B.LS_BF16, 0, 100, 100, A, 1e-3, A, A, 0, None, A, A, None, A, 100,
                                 None) == B.LS_OK
