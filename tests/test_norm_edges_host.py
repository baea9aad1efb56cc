"""Host-side bounds of the row norm's arguments (no GPU needed)."""
import ctypes

import pytest

import farthest_vector_search_amd as vs

SHAPE = 2


@pytest.mark.parametrize("eps,status", [(0.0, 0), (1e-45, 0), (3.4e38, 0), (3.4028234e38, 0),
                                        (-1e-45, SHAPE), (float("inf"), SHAPE), (float("nan"), SHAPE)])
def test_every_finite_eps_is_taken(eps, status):
    P = ctypes.c_void_p
    L = vs.lib()
    assert L.vs_norm_rows(P(0), None, None, 0, 8, 0, eps, None, P(0), None, None) == status
    assert L.vs_norm_rows_q8(P(0), None, None, 0, 8, 0, eps, None, P(0), P(0), None) == status
