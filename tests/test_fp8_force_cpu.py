"""The product's test switches: what they refuse (no GPU; nothing is launched)."""
import ctypes

import pytest

from bit_quantization_aware_b200 import build as pqbuild


@pytest.fixture(scope="module")
def pq():
    pqbuild.build()
    from bit_quantization_aware_b200 import pq
    pq.lib()
    yield pq
    pq.pq_debug_fp8_force(0, 0)


def test_force_refusals(pq):
    for bad in ((64, 0), (0, 1), (32, 1), (256, 2), (128, 3), (64, 16), (-64, 1), (64, -1)):
        with pytest.raises(pq.PQError):
            pq.pq_debug_fp8_force(*bad)
    for good in ((64, 8), (128, 4), (256, 1)):
        pq.pq_debug_fp8_force(*good)
        assert pq.pq_debug_fp8_choice(5, 70, 2000, pq.PQ_BLOCK_TILE) == good
    pq.pq_debug_fp8_force(128, 1)
    with pytest.raises(pq.PQError):
        pq.pq_debug_fp8_choice(5, 70, 2000, pq.PQ_BLOCK_ROW)
    pq.pq_debug_fp8_force(64, 8)
    with pytest.raises(pq.PQError):  # seven K blocks
        pq.pq_debug_fp8_choice(5, 70, 896, pq.PQ_BLOCK_ROW)


def test_choice_refusals(pq):
    f, w = pq.lib().pq_debug_fp8_choice, ctypes.c_int()
    r = ctypes.byref(w)
    for args in ((0, 1, 1, 2, r, r), (1, 0, 1, 2, r, r), (1, 1, 0, 2, r, r), (1, 1, 1, 3, r, r), (1, 1, 1, 2, None, r),
                 (1, 1, 1, 2, r, None)):
        assert f(*args) == pq.PQ_ERR_INVALID_ARG
