"""Host side of clipping in the step classes: which buffers the norm calls use
and what they are told to write (nothing is launched; no GPU)."""
import pytest
import torch

from bit_quantization_aware_b200 import build as pqbuild
from bit_quantization_aware_b200 import inputs as I
from bit_quantization_aware_b200.sharded import LocalPeers, ShardedQuantStep
from tests.test_sharded_clip_cpu import ClipLib

MATS = [I.Matrix("a", 16, 64, 0, 0), I.Matrix("b", 5, 24, 0, 1), I.Matrix("none", 0, 8, 0, 2)]


@pytest.fixture()
def pq(monkeypatch):
    """The binding with CPU tensors in its descriptors and no launches."""
    pqbuild.build()
    from bit_quantization_aware_b200 import pq
    pq.calls = []
    monkeypatch.setattr(pq, "matrix_array", list)
    monkeypatch.setattr(pq, "tensor_array", lambda ts, outs=None: list(ts))
    monkeypatch.setattr(pq, "pq_grad_norm", lambda *a, **k: pq.calls.append((a, k)))
    monkeypatch.setattr(pq, "pq_grad_clip", lambda *a: pq.calls.append((a, {})))
    yield pq
    del pq.calls


def step(pq, **kw):
    from bit_quantization_aware_b200.step import QuantStep
    return QuantStep(MATS, pq.PQ_SEQ2, device="cpu", **kw)


def no_new_memory(monkeypatch):
    def refuse(*a, **k):
        raise AssertionError("memory made inside a call belongs to the current stream, not to the call's")
    for name in ("empty", "zeros", "ones", "full", "tensor"):
        monkeypatch.setattr(torch, name, refuse)


def test_quant_step_makes_its_norm_buffers_when_it_is_made(pq, monkeypatch):
    st = step(pq)
    no_new_memory(monkeypatch)
    st.grad_norm(1.0, stream=77)
    st.clip_grads(1.0, stream=77)
    (norm, _), (clip, _) = pq.calls
    assert norm[3].numel() >= pq.pq_grad_norm_workspace_bytes(0, len(MATS))
    assert clip[4].numel() >= pq.pq_grad_norm_workspace_bytes(len(clip[0]), 0)
    bufs = [norm[1], norm[2], norm[3], clip[2], clip[3], clip[4]]
    assert len({t.data_ptr() for t in bufs}) == len(bufs)


def test_sharded_step_makes_its_norm_buffers_when_it_is_made(monkeypatch):
    mats = [I.Matrix("a", 16, 64, 0, 0)]
    st = ShardedQuantStep(mats, 3, 0, 1, LocalPeers(1), device="cpu", lib=ClipLib)
    st.g(0).fill_(1.0)
    with monkeypatch.context() as m:
        m.setattr(ClipLib, "pq_reduce_grad_norm", staticmethod(lambda *a, sumsq_out, stream: sumsq_out.fill_(4.0)))
        no_new_memory(m)
        norm, coef = st.clip_coef(1.0, stream=77)
    assert float(norm) == 2.0



def test_quant_step_norm_writes_no_gradient(pq):
    st = step(pq)
    st.grad_norm(1.0)
    mats = pq.calls[0][1]["mats"]
    assert [m["g"].data_ptr() for m in mats] == [b.g.data_ptr() for b in st.bufs]
    assert all(m.get("dalpha") is None and m.get("dw") is None for m in mats)


def test_clipping_without_outputs_is_refused(pq):
    st = step(pq, alloc_outputs=False)
    with pytest.raises(ValueError, match="alloc_outputs"):
        st.clip_grads(1.0)
    st.grad_norm(1.0)  # which needs none
    assert len(pq.calls) == 1


def test_other_parameters_count_through_gather():
    """Sums behind the ranks' enter the norm and the factor."""
    mats = [I.Matrix("a", 16, 64, 0, 0)]
    st = ShardedQuantStep(mats, 3, 0, 1, LocalPeers(1), device="cpu", lib=ClipLib)
    st.g(0).fill_(0.5)  # 256 in squares
    other = torch.tensor([900.0, 69.0], dtype=torch.float64)
    norm = st.backward(lambda: None, None, None, max_norm=7.0, gather=lambda mine: torch.cat([mine, other]))
    assert float(norm) == 35.0
    assert torch.allclose(st.w_shard(0), torch.full((16, 64), 0.5 * 7 / 35), rtol=2.0 ** -22, atol=0)
