"""Pointers that are not aligned to their element are refused on the host by
every call around the training step: a kernel that took one would fault (no
GPU; nothing is launched)."""
import ctypes

import pytest

from bit_quantization_aware_b200 import build as pqbuild

AT = 0x10000  # never dereferenced: rejected on the host


@pytest.fixture(scope="module")
def pq():
    pqbuild.build()
    from bit_quantization_aware_b200 import pq
    pq.lib()
    return pq


def p(offset=0):
    return ctypes.c_void_p(AT + offset)


@pytest.fixture()
def refused(pq):
    n0 = pq.pq_launch_count()
    yield lambda status: status == pq.PQ_ERR_MISALIGNED
    assert pq.pq_launch_count() == n0


@pytest.mark.parametrize("off", [1, 2, 3])
def test_scales(pq, refused, off):
    quant = lambda s, st: pq.lib().pq_fp8_quant(pq.PQ_BLOCK_ROW, pq.PQ_BF16, 4, 8, p(), 8, p(), 16, s, p(), 16, st, None)
    assert refused(quant(p(off), p())) and refused(quant(p(), p(off)))
    for block in (pq.PQ_BLOCK_ROW, pq.PQ_BLOCK_TILE):
        gemm = lambda sa, sb: pq.lib().pq_fp8_gemm(4, 8, 32, p(), 32, sa, p(), 32, sb, block, p(), pq.PQ_BF16, 8, None)
        assert refused(gemm(p(off), p())) and refused(gemm(p(), p(off)))


def outputs(off):
    """(sumsq, norm, coef) with one of them off its element's alignment."""
    return [(p(off), p(), p()), (None, p(off % 4 or 1), p()), (None, p(), p(off % 4 or 1))]


@pytest.mark.parametrize("off", [1, 2, 4])
def test_norms_and_factors(pq, refused, off):
    L, need = pq.lib(), pq.pq_grad_norm_workspace_bytes(1, 1)
    one = (pq.PQTensor * 1)(pq.PQTensor(AT, 10, None, pq.PQ_FP32, 0))
    shard = pq.shard_array([dict(rows=2, cols=8, w=AT, alpha=AT)])
    srcs = (ctypes.c_void_p * 1)(AT)
    for sq, no, co in outputs(off):
        assert refused(L.pq_grad_norm(1, one, 0, 0, None, 1.0, sq, no, co, p(), need, None))
        assert refused(L.pq_reduce_grad_norm(pq.PQ_SEQ2, 1, srcs, 1.0, 1, shard, 1.0, sq, no, co, p(), need, None))
        assert refused(L.pq_clip_coef(1, sq or p(), 1.0, no, co, None))
    for _, no, co in outputs(off)[1:]:
        assert refused(L.pq_grad_clip(1, one, 1.0, no, co, p(), need, None))


@pytest.mark.parametrize("off", [1, 2, 3])
def test_factors_that_are_read(pq, refused, off):
    L, hp = pq.lib(), pq.adamw(1, 1e-3)
    one = (pq.PQTensor * 1)(pq.PQTensor(AT, 10, None, pq.PQ_FP32, 0))
    assert refused(L.pq_grad_scale(1, one, p(off), None))
    mats, shards = pq.adamw_matrix_array([]), pq.shard_array([])
    srcs = (ctypes.c_void_p * 1)(AT)
    h = ctypes.byref(hp)
    assert refused(L.pq_fakequant_bwd_adamw_clip(pq.PQ_SEQ2, 0, mats, h, h, p(off), None))
    assert refused(L.pq_reduce_bwd_adamw_clip(pq.PQ_SEQ2, 1, srcs, 1.0, 0, shards, h, h, p(off), None))


@pytest.mark.parametrize("key,off", [("w", 2), ("w", 1), ("alpha", 2), ("dalpha", 3), ("g", 1)])
def test_matrices_and_shards_of_a_norm(pq, refused, key, off):
    L, need = pq.lib(), pq.pq_grad_norm_workspace_bytes(0, 1)
    mat = dict(rows=2, cols=8, w=AT, alpha=AT, g=AT, dalpha=AT)
    mat[key] += off
    assert refused(L.pq_grad_norm(0, None, pq.PQ_SEQ2, 1, pq.matrix_array([mat]), 1.0, None, p(), None, p(), need, None))
    shard = dict(rows=2, cols=8, w=AT, alpha=AT, dalpha=AT)
    srcs = (ctypes.c_void_p * 1)(AT + off if key == "g" else AT)
    if key != "g":
        shard[key] += off
    assert refused(L.pq_reduce_grad_norm(pq.PQ_SEQ2, 1, srcs, 1.0, 1, pq.shard_array([shard]), 1.0, None, p(), None,
                                         p(), need, None))
