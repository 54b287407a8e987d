"""Argument checks of the e4m3 block calls and of the gradient norm and
clipping calls, and their host-side helpers: nothing is launched (no GPU)."""
import ctypes

import pytest
import torch

from bit_quantization_aware_b200 import build as pqbuild
from tests import fp8_ref as R


@pytest.fixture(scope="module")
def pq():
    pqbuild.build()
    from bit_quantization_aware_b200 import pq
    pq.lib()
    return pq


FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: rejected on the host
ODD = ctypes.c_void_p(0x10001)


def test_quant_refusals(pq):
    f = pq.lib().pq_fp8_quant
    E, M = pq.PQ_ERR_INVALID_ARG, pq.PQ_ERR_MISALIGNED
    good = [pq.PQ_BLOCK_ROW, pq.PQ_BF16, 4, 8, FAKE, 8, FAKE, 16, FAKE, FAKE, 16, FAKE, None]

    def bad(status, **kw):
        names = ("block", "dtype", "rows", "cols", "x", "ldx", "q", "ldq", "s", "qt", "ldqt", "st", "stream")
        args = dict(zip(names, good))
        args.update(kw)
        n0 = pq.pq_launch_count()
        assert f(*args.values()) == status, kw
        assert pq.pq_launch_count() == n0

    for kw in (dict(block=0), dict(block=3), dict(dtype=0), dict(dtype=4), dict(rows=-1), dict(cols=-1),
               dict(x=None), dict(ldx=7), dict(ldq=7), dict(ldqt=3), dict(q=None), dict(s=None), dict(qt=None),
               dict(st=None), dict(q=None, s=None, qt=None, st=None)):
        bad(E, **kw)
    bad(M, x=ODD)
    bad(M, x=ctypes.c_void_p(0x10002), dtype=pq.PQ_FP32)
    bad(pq.PQ_OK, rows=0, x=None)
    bad(pq.PQ_OK, cols=0, x=None, ldx=0)
    bad(pq.PQ_ERR_UNSUPPORTED, rows=1 << 40, cols=1 << 20, ldx=1 << 20, ldq=1 << 20, ldqt=1 << 40)


def test_product_refusals(pq):
    f = pq.lib().pq_fp8_gemm
    E, M = pq.PQ_ERR_INVALID_ARG, pq.PQ_ERR_MISALIGNED
    names = ("m", "n", "k", "a", "lda", "sa", "b", "ldb", "sb", "block", "y", "dtype", "ldy", "stream")
    good = [4, 8, 32, FAKE, 32, FAKE, FAKE, 32, FAKE, pq.PQ_BLOCK_TILE, FAKE, pq.PQ_BF16, 8, None]

    def bad(status, **kw):
        args = dict(zip(names, good))
        args.update(kw)
        n0 = pq.pq_launch_count()
        assert f(*args.values()) == status, kw
        assert pq.pq_launch_count() == n0

    for kw in (dict(m=-1), dict(n=-1), dict(k=-1), dict(a=None), dict(b=None), dict(sa=None), dict(sb=None),
               dict(y=None), dict(block=0), dict(dtype=0), dict(lda=16), dict(ldb=16), dict(ldy=7)):
        bad(E, **kw)
    for kw in (dict(a=ODD), dict(b=ctypes.c_void_p(0x10008)), dict(lda=40), dict(ldb=33), dict(y=ODD),
               dict(y=ctypes.c_void_p(0x10002), dtype=pq.PQ_FP32)):
        bad(M, **kw)
    bad(pq.PQ_OK, m=0, a=None)
    bad(pq.PQ_OK, n=0, b=None, ldy=0)
    bad(pq.PQ_ERR_UNSUPPORTED, m=1 << 31)


def test_norm_and_clip_refusals(pq):
    L, E, M = pq.lib(), pq.PQ_ERR_INVALID_ARG, pq.PQ_ERR_MISALIGNED
    need = pq.pq_grad_norm_workspace_bytes(1, 1)
    assert need > 0 and pq.pq_grad_norm_workspace_bytes(-1, 0) == -1 == pq.pq_grad_norm_workspace_bytes(0, -1)

    def tensor(data=0x10000, numel=10, out=None, dtype=pq.PQ_FP32, out_dtype=0):
        return (pq.PQTensor * 1)(pq.PQTensor(data, numel, out, dtype, out_dtype))

    def mat(**kw):
        d = dict(rows=2, cols=8, w=0x10000, alpha=0x10000, g=0x10000, grad_scale=1.0)
        d.update(kw)
        return pq.matrix_array([d])

    n0 = pq.pq_launch_count()
    norm = lambda n=1, t=tensor(), q=pq.PQ_SEQ2, nm=1, m=mat(), mx=1.0, sq=None, no=FAKE, co=None, ws=FAKE, b=need: \
        L.pq_grad_norm(n, t, q, nm, m, mx, sq, no, co, ws, b, None)
    for kw in (dict(n=-1), dict(n=1, t=None), dict(nm=-1), dict(nm=1, m=None), dict(q=0), dict(q=9), dict(mx=-1.0),
               dict(mx=float("nan")), dict(no=None), dict(ws=None), dict(b=need - 1), dict(ws=ctypes.c_void_p(0x10004)),
               dict(t=tensor(data=None)), dict(t=tensor(numel=-1)), dict(t=tensor(dtype=0)), dict(t=tensor(dtype=4)),
               dict(m=mat(rows=-1)), dict(m=mat(cols=-1)), dict(m=mat(w=None)), dict(m=mat(alpha=None)),
               dict(m=mat(g=None))):
        assert norm(**kw) == E, kw
    assert norm(t=tensor(data=0x10002)) == M
    assert norm(t=tensor(data=0x10001, dtype=pq.PQ_BF16)) == M

    clip = lambda t=tensor(), mx=1.0, no=FAKE, ws=FAKE, b=need: L.pq_grad_clip(1, t, mx, no, None, ws, b, None)
    for kw in (dict(mx=-0.5), dict(no=None), dict(ws=None), dict(b=8),
               dict(t=tensor(out=0x20000, out_dtype=pq.PQ_BF16)), dict(t=tensor(out=0x20000, out_dtype=0)),
               dict(t=tensor(dtype=pq.PQ_BF16, out=0x20000, out_dtype=pq.PQ_FP16))):
        assert clip(**kw) == E, kw
    assert clip(t=tensor(out=0x20002, out_dtype=pq.PQ_FP32)) == M
    assert L.pq_grad_scale(1, tensor(), None, None) == E
    assert L.pq_grad_scale(-1, None, FAKE, None) == E
    assert L.pq_grad_scale(0, None, FAKE, None) == pq.PQ_OK
    assert L.pq_clip_coef(-1, FAKE, 1.0, FAKE, FAKE, None) == E
    assert L.pq_clip_coef(1, None, 1.0, FAKE, FAKE, None) == E
    assert L.pq_clip_coef(1, FAKE, 1.0, None, None, None) == E

    shard = pq.shard_array([dict(rows=2, cols=8, w=0x10000, alpha=0x10000)])
    srcs = (ctypes.c_void_p * 17)(*[0x10000] * 17)
    red = lambda q=pq.PQ_SEQ2, ns=1, s=srcs, n=1, sh=shard, mx=1.0, sq=FAKE, ws=FAKE: \
        L.pq_reduce_grad_norm(q, ns, s, 1.0, n, sh, mx, sq, None, None, ws, need, None)
    for kw in (dict(q=0), dict(ns=0), dict(ns=17), dict(s=None), dict(n=-1), dict(sh=None), dict(mx=-1.0),
               dict(sq=None), dict(ws=None), dict(s=(ctypes.c_void_p * 1)(None))):
        assert red(**kw) == E, kw

    hp = pq.adamw(1, 1e-3)
    one = pq.adamw_matrix_array([dict(rows=1, cols=8)])
    assert L.pq_fakequant_bwd_adamw_clip(pq.PQ_SEQ2, 1, one, ctypes.byref(hp), ctypes.byref(hp), None, None) == E
    assert L.pq_reduce_bwd_adamw_clip(pq.PQ_SEQ2, 1, srcs, 1.0, 1, shard, ctypes.byref(hp), ctypes.byref(hp), None,
                                      None) == E
    assert pq.pq_launch_count() == n0


class FakeCuda:
    """Stands for a CUDA tensor in host-side checks."""

    is_cuda = True

    def __init__(self, t, at=0x10000):
        self.t, self.at = t, at

    def data_ptr(self):
        return self.at

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refusals(pq):
    t = lambda n=8, dtype=torch.float32, at=0x10000: FakeCuda(torch.zeros(n, dtype=dtype), at)
    with pytest.raises(ValueError, match="bf16, fp16 or fp32"):
        pq.tensor_array([t(dtype=torch.float64)])
    with pytest.raises(ValueError, match="CUDA"):
        pq.tensor_array([torch.zeros(3)])
    with pytest.raises(ValueError, match="contiguous"):
        pq.tensor_array([FakeCuda(torch.zeros(4, 4)[:, :2])])
    with pytest.raises(ValueError, match="same tensor"):
        pq.tensor_array([t(), t()])
    with pytest.raises(ValueError, match="one entry"):
        pq.tensor_array([t()], [])
    with pytest.raises(ValueError, match="size and its type"):
        pq.tensor_array([t()], [t(7)])
    with pytest.raises(ValueError, match="size and its type"):
        pq.tensor_array([t()], [t(8, torch.bfloat16)])
    arr = pq.tensor_array([t(dtype=torch.bfloat16), t(at=0x20000)], [t(at=0x30000), None])
    assert [(a.dtype, a.out, a.out_dtype, a.numel) for a in arr] == [(pq.PQ_BF16, 0x30000, pq.PQ_FP32, 8),
                                                                     (pq.PQ_FP32, None, 0, 8)]
    with pytest.raises(ValueError, match="one torch.float32"):
        pq.pq_grad_norm(1.0, t(2), None, t(at=0x50000), tensors=arr)
    with pytest.raises(ValueError, match="one torch.float64"):
        pq.pq_grad_norm(1.0, None, None, t(at=0x50000), tensors=arr, sumsq_out=t(1))
    with pytest.raises(ValueError, match="at least one"):
        pq.clip_grad_norm([], 1.0)

    m = lambda r, c, dtype=torch.float32: FakeCuda(torch.zeros(r, c, dtype=dtype))
    u8 = torch.uint8
    with pytest.raises(ValueError, match="x must be a matrix"):
        pq.pq_fp8_quant(1, m(4, 8, torch.float64))
    with pytest.raises(ValueError, match="contiguous rows"):
        pq.pq_fp8_quant(1, FakeCuda(torch.zeros(8, 4).t()))
    with pytest.raises(ValueError, match=r"q_out must be \[4, 8\]"):
        pq.pq_fp8_quant(1, m(4, 8), m(4, 9, u8), m(1, 4))
    with pytest.raises(ValueError, match=r"scales of q_out must be fp32 \[1, 4\]"):
        pq.pq_fp8_quant(1, m(4, 8), m(4, 8, u8), m(4, 1))
    with pytest.raises(ValueError, match=r"scales of qt_out must be fp32 \[1, 8\]"):
        pq.pq_fp8_quant(1, m(4, 8), qt_out=m(8, 4, u8), st_out=m(1, 4))
    with pytest.raises(ValueError, match="block"):
        pq.pq_fp8_quant(3, m(4, 8), m(4, 8, u8), m(4, 1))
    with pytest.raises(ValueError, match="shapes"):
        pq.pq_fp8_gemm(m(4, 32, u8), m(1, 4), m(8, 48, u8), m(1, 1), 2, m(4, 8))
    with pytest.raises(ValueError, match="a_scale"):
        pq.pq_fp8_gemm(m(4, 32, u8), m(4, 1), m(8, 32, u8), m(1, 1), 2, m(4, 8))
    with pytest.raises(ValueError, match="b_scale"):
        pq.pq_fp8_gemm(m(4, 32, u8), m(1, 4), m(8, 32, u8), m(1, 8), 2, m(4, 8))
    with pytest.raises(ValueError, match="overlap"):
        pq.pq_fp8_gemm(FakeCuda(torch.zeros(1, 32, dtype=u8).expand(4, 32)), m(1, 4), m(8, 32, u8), m(1, 1), 2, m(4, 8))


def test_tensors_of_another_device_are_refused(pq, monkeypatch):
    """One device a call, and the current one: its stream launches."""
    class On(FakeCuda):
        def __init__(self, dev, *shape, dtype=torch.float32):
            super().__init__(torch.zeros(*shape, dtype=dtype))
            self.dev = dev

        def get_device(self):
            return self.dev

    monkeypatch.setattr(pq, "_current_device", lambda: 0)
    u8 = torch.uint8
    for a, b, word in ((0, 1, "different devices"), (1, 1, "current device is cuda:0")):
        with pytest.raises(ValueError, match=word):
            pq.pq_fp8_gemm(On(a, 4, 32, dtype=u8), On(b, 1, 4), On(b, 8, 32, dtype=u8), On(b, 1, 1), 2, On(b, 4, 8))
        with pytest.raises(ValueError, match=word):
            pq.pq_fp8_quant(1, On(a, 4, 8), On(b, 4, 8, dtype=u8), On(b, 1, 4))
        with pytest.raises(ValueError, match=word):
            pq.tensor_array([On(a, 8), On(b, 8)])
        with pytest.raises(ValueError, match=word):
            pq.pq_clip_coef(On(a, 1, dtype=torch.float64), 1.0, On(b, 1), On(b, 1))
    arr = pq.tensor_array([On(0, 8)])
    with pytest.raises(ValueError, match="different devices"):
        pq.pq_grad_clip(arr, 1.0, On(1, 1), None, On(1, 64, dtype=u8))
    with pytest.raises(ValueError, match="different devices"):
        pq.pq_grad_scale(arr, On(1, 1))
    with pytest.raises(ValueError, match="different devices"):
        pq.pq_grad_norm(1.0, On(1, 1), None, On(1, 64, dtype=u8), tensors=arr)


def test_linear_refusals(pq, monkeypatch):
    from bit_quantization_aware_b200.linear import Fp8Linear
    monkeypatch.setattr(pq, "pq_fp8_quant", lambda *a: None)
    monkeypatch.setattr(pq, "pq_fp8_gemm", lambda *a: None)
    with pytest.raises(ValueError, match="positive"):
        Fp8Linear(0, 4, 4, device="cpu")
    layer = Fp8Linear(6, 4, 5, device="cpu")
    with pytest.raises(ValueError, match="forward first"):
        layer.backward(torch.zeros(2, 6))
    for x, w in ((torch.zeros(6, 4), torch.zeros(6, 4)), (torch.zeros(0, 4), torch.zeros(6, 4)),
                 (torch.zeros(2, 3), torch.zeros(6, 4)), (torch.zeros(2, 4), torch.zeros(4, 6))):
        with pytest.raises(ValueError):
            layer.forward(x, w)
    assert layer.forward(torch.zeros(2, 4), torch.zeros(6, 4)).shape == (2, 6)
    with pytest.raises(ValueError, match="dy"):
        layer.backward(torch.zeros(3, 6))
    dx, dw = layer.backward(torch.zeros(2, 6))
    assert dx.shape == (2, 4) and dw.shape == (6, 4)


def test_scale_shapes_and_pitches(pq):
    assert pq.fp8_scale_shape(pq.PQ_BLOCK_ROW, 5, 129) == (2, 5)
    assert pq.fp8_scale_shape(pq.PQ_BLOCK_TILE, 129, 128) == (2, 1)
    q = pq.fp8_empty(3, 17, "cpu")
    assert q.shape == (3, 17) and q.stride() == (32, 1) and q.dtype == torch.float8_e4m3fn


def test_reference_rounding_is_e4m3():
    """The 64-bit reference's rounding against torch's conversion of every
    e4m3 value, the midpoints between neighbours and values beside them."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    v = torch.cat([v, -v])
    assert torch.equal(R.e4m3(v), v.float().to(torch.float8_e4m3fn).double())
    assert torch.equal(R.e4m3(torch.tensor([1e6, -500.0, 448.1], dtype=torch.float64)),
                       torch.tensor([448.0, -448.0, 448.0], dtype=torch.float64))


def test_overlapping_gradients_are_refused(pq):
    """Units are scaled in any order, so no entry may write memory that another
    one, or its own input, uses."""
    t = lambda at, n=8, dtype=torch.float32: FakeCuda(torch.zeros(n, dtype=dtype), at)
    A, B = 0x10000, 0x10020  # B is right behind eight fp32 values at A
    ok = [([t(A), t(B)], None), ([t(A)], [t(A)]), ([t(A), t(A)], [t(B), t(0x20000)]),
          ([t(A, 8, torch.bfloat16)], [t(A + 16)]), ([t(A, 0), t(A)], None)]
    for tensors, outs in ok:
        assert len(pq.tensor_array(tensors, outs)) == len(tensors)
    bad = [([t(A), t(A + 16)], None),                  # views that share half
           ([t(A, 64), t(B), t(0x20000)], None),       # one inside another
           ([t(A), t(B)], [t(B), t(0x20000)]),         # an out over another's data
           ([t(A), t(B)], [t(0x20000), t(0x20010)]),   # outs that share half
           ([t(A)], [t(A + 4)]),                       # its own data, shifted
           ([t(A, 8, torch.bfloat16)], [t(A)])]        # fp32 over its own bf16 data
    for tensors, outs in bad:
        with pytest.raises(ValueError, match="two entries"):
            pq.tensor_array(tensors, outs)
    for dtype, at in ((pq.PQ_FP32, A + 4), (pq.PQ_BF16, A), (pq.PQ_BF16, A + 12), (pq.PQ_FP32, A - 28)):
        arr = (pq.PQTensor * 1)(pq.PQTensor(A, 8, at, dtype, pq.PQ_FP32))
        assert pq.lib().pq_grad_scale(1, arr, FAKE, None) == pq.PQ_ERR_INVALID_ARG, (dtype, at)


def test_linear_forgets_a_forward_that_another_broke_into(pq, monkeypatch):
    """A forward that fails halfway has overwritten the weights' codes of the
    one before: backward refuses instead of mixing the two."""
    from bit_quantization_aware_b200.linear import Fp8Linear
    monkeypatch.setattr(pq, "pq_fp8_quant", lambda *a: None)
    monkeypatch.setattr(pq, "pq_fp8_gemm", lambda *a: None)
    layer = Fp8Linear(6, 4, 5, device="cpu")
    x, w, dy = torch.zeros(2, 4), torch.zeros(6, 4), torch.zeros(2, 6)
    layer.forward(x, w)
    with pytest.raises(ValueError):  # refused before anything is written: the last forward stands
        layer.forward(torch.zeros(2, 3), w)
    layer.backward(dy)

    def refuse(*a):
        raise ValueError("y_out")

    monkeypatch.setattr(pq, "pq_fp8_gemm", refuse)
    with pytest.raises(ValueError, match="y_out"):
        layer.forward(x, w)
    monkeypatch.setattr(pq, "pq_fp8_gemm", lambda *a: None)
    with pytest.raises(ValueError, match="forward first"):
        layer.backward(dy)
    layer.forward(x, w)
    layer.backward(dy)


def test_clipping_factors_of_another_device_are_refused(pq, monkeypatch):
    class On(FakeCuda):
        def __init__(self, dev, *shape, dtype=torch.float32):
            super().__init__(torch.zeros(*shape, dtype=dtype))
            self.dev = dev

        def get_device(self):
            return self.dev

    monkeypatch.setattr(pq, "_current_device", lambda: 0)
    hp = pq.adamw(1, 1e-3)
    n0 = pq.pq_launch_count()
    with pytest.raises(ValueError, match="current device is cuda:0"):
        pq.pq_fakequant_bwd_adamw(pq.PQ_SEQ2, pq.adamw_matrix_array([]), hp, hp, coef=On(1, 1))
    with pytest.raises(ValueError, match="current device is cuda:0"):
        pq.pq_reduce_bwd_adamw(pq.PQ_SEQ2, [0x10000], 1.0, pq.shard_array([]), hp, hp, coef=On(1, 1))
    with pytest.raises(ValueError, match="different devices"):
        pq.pq_reduce_grad_norm(pq.PQ_SEQ2, [0x10000], 1.0, pq.shard_array([]), 1.0, On(0, 1), None,
                               On(1, 64, dtype=torch.uint8))
    assert pq.pq_launch_count() == n0
