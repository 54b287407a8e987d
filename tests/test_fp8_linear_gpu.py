"""What the e4m3 linear layer multiplies by, and how far its products may be
from those of the operands that it was given."""
import pytest
import torch

from tests import fp8_ref as R
from tests.test_fp8_gpu import DEV, draw, pq  # noqa: F401 (pq is a fixture)

pytestmark = pytest.mark.gpu


def moved(t, block):
    """The most that each value of t moves when it becomes an e4m3 code: half a
    step, 2^-4 of the value, or half of the smallest step, 2^-10 scales. The
    scale, the factor and the product in front of the rounding are off by
    2^-24 each, together less than 2^-4 * 2^-18 of the value."""
    a = R.amax(t.float(), block).double()
    return torch.maximum(t.double().abs() * 2.0 ** -4, R.expand(a / 448.0, block, *t.shape) * 2.0 ** -10) * (1 + 2.0 ** -18)


@pytest.mark.parametrize("qname", ["ternary", "seq2", "lsq3", "lsq4"])
def test_products_of_rounded_operands(pq, qname):  # noqa: F811
    """Every operand is rounded to e4m3 once, the fake-quantized weights among
    them: products are within the roundings of both."""
    from bit_quantization_aware_b200 import inputs as I
    from bit_quantization_aware_b200.linear import Fp8Linear
    m, n, k = 70, 264, 400
    q = pq.QUANTIZERS[qname]
    w = I.normal_weights(n, k, seed=1, stream=0, device=DEV)
    wq, _ = pq.fakequant_fwd(q, w, I.alpha_init(w, q))
    x, dy = draw(m, k, 1, torch.bfloat16), draw(m, n, 2, torch.bfloat16, 1e-3)
    layer = Fp8Linear(n, k, m, device=DEV)
    f32 = lambda *s: torch.empty(*s, device=DEV)
    y = layer.forward(x.to(DEV), wq, f32(m, n))
    dx, dw = layer.backward(dy.to(DEV), f32(m, k), f32(n, k))
    wq = wq.cpu()
    cols = lambda t: moved(t.t().contiguous(), R.ROW).t()
    ops = {"y": (y, x, wq.t(), moved(x, R.ROW), moved(wq, R.TILE).t()),
           "dx": (dx, dy, wq, moved(dy, R.ROW), moved(wq, R.TILE)),
           "dw": (dw, dy.t(), x, cols(dy).t(), cols(x))}
    for name, (got, a, b, da, db) in ops.items():
        a, b = a.double(), b.double()
        err = (got.cpu().double() - a @ b).abs()
        mags = (a.abs() + da) @ (b.abs() + db)
        # rounding of the operands, and the product's own sums (fp8_ref)
        tol = mags - a.abs() @ b.abs() + R.product_tolerance(mags, mags, a.shape[1], torch.float32)
        assert (err <= tol).all(), name
    # the weights do move: the rows' scales put their levels between the codes of a tile
    rms = ((R.values(*_codes(wq), R.TILE) - wq.double()).square().sum() / wq.double().square().sum()).sqrt()
    assert 0 < float(rms) <= 2.0 ** -4


def _codes(t):
    v, s = R.quant(t, R.TILE)
    return v.float().to(torch.float8_e4m3fn), s
