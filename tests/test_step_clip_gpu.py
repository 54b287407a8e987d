"""Clipping in the step classes on the GPU: streams of their own, and what a
norm leaves untouched."""
import pytest
import torch

from bit_quantization_aware_b200 import inputs as I
from tests.test_grad_norm_gpu import DEV, RTOL, coef_of, norm64, pq  # noqa: F401 (pq is a fixture)

pytestmark = pytest.mark.gpu

MATS = [I.Matrix("a", 256, 512, 0, 0), I.Matrix("b", 33, 72, 0, 1)]


def backlog():
    """A tenth of a second or so of work on the current stream."""
    t = torch.zeros(1 << 28, device=DEV)
    for _ in range(200):
        t.add_(1.0)
    return t


@pytest.mark.parametrize("as_int", [False, True])
def test_first_calls_on_another_stream(pq, as_int):  # noqa: F811
    """Nothing of a first call waits in the current stream's queue, where it
    would land on the results."""
    from bit_quantization_aware_b200.step import QuantStep
    st = QuantStep(MATS, pq.PQ_SEQ2, device=DEV)
    st.generate(seed=3)
    st.run()
    want = norm64([t for b in st.bufs for t in (b.dw, b.dalpha)])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = backlog()
    stream = side.cuda_stream if as_int else side
    norm, coef = st.grad_norm(0.25 * want, stream)
    clipped = st.clip_grads(0.25 * want, stream)
    side.synchronize()
    with torch.cuda.stream(side):
        early = [float(t) for t in (norm, coef, clipped)]
    torch.cuda.synchronize()
    del busy
    assert [float(t) for t in (norm, coef, clipped)] == early
    assert early[0] == pytest.approx(want, rel=RTOL) and early[2] == pytest.approx(want, rel=RTOL)
    assert early[1] == pytest.approx(coef_of(want, 0.25 * want), rel=RTOL)


def test_first_sharded_norm_on_another_stream(pq):  # noqa: F811
    from bit_quantization_aware_b200.sharded import LocalPeers, ShardedQuantStep
    st = ShardedQuantStep(MATS, pq.PQ_LSQ4, 0, 1, LocalPeers(1), device=DEV)
    grads = []
    for i, m in enumerate(MATS):
        w = I.normal_weights(m.rows, m.cols, seed=i, stream=0, device=DEV)
        a = I.alpha_init(w, pq.PQ_LSQ4)
        g = I.grad_bf16(m.rows, m.cols, seed=9, stream=i, device=DEV)
        st.load_full(i, w, a)
        st.g(i).copy_(g)
        grads += pq.fakequant_bwd(pq.PQ_LSQ4, w, a, g, pq.pq_default_grad_scale(pq.PQ_LSQ4, m.cols))
    want = norm64(grads)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = backlog()
    norm, coef = st.clip_coef(0.25 * want, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        early = float(norm), float(coef)
    torch.cuda.synchronize()
    del busy
    assert (float(norm), float(coef)) == early
    assert early[0] == pytest.approx(want, rel=RTOL)
    assert early[1] == pytest.approx(coef_of(want, 0.25 * want), rel=RTOL)


def test_norm_after_clipping_leaves_the_clipped_gradients(pq):  # noqa: F811
    from bit_quantization_aware_b200.step import QuantStep
    st = QuantStep(MATS, pq.PQ_SEQ2, device=DEV)
    st.generate(seed=3)
    st.run()
    first = float(st.grad_norm(1.0)[0])
    st.clip_grads(0.25 * first)
    clipped = [t.clone() for b in st.bufs for t in (b.dw, b.dalpha)]
    again, _ = st.grad_norm(1.0)  # for a log, say: that of the unclipped gradient
    assert float(again) == first
    for t, k in zip([t for b in st.bufs for t in (b.dw, b.dalpha)], clipped):
        assert torch.equal(t, k)
