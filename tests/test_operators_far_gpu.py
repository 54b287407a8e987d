"""Block quantization, products, norms and clipping where offsets pass 32
bits, and products of narrow and of very deep operands."""
import math

import pytest
import torch

from tests import fp8_ref as R
from tests.test_fp8_gpu import DEV, check_product, draw, pq, same_codes  # noqa: F401 (pq is a fixture)
from tests.test_grad_norm_gpu import RTOL, coef_of, outs, scratch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [R.TILE, R.ROW])
@pytest.mark.parametrize("m,n,k", [(1, 300, 14336), (77, 515, 14336), (2100, 2049, 14336), (40, 8, 200), (300, 24, 300),
                                   (2500, 2056, 16)])
def test_narrow_and_deep_products(pq, m, n, k, block):  # noqa: F811
    check_product(pq, m, n, k, block, "bf16", seed=m + n)


@pytest.mark.parametrize("block", [R.TILE, R.ROW])
def test_rows_far_apart(pq, block):  # noqa: F811
    """Rows 2^27 elements apart: the last begins behind 2^31 of them."""
    rows, cols, pitch = 20, 264, 1 << 27
    x = draw(rows, cols, 1, torch.bfloat16).to(DEV)
    w = draw(50, cols, 2).to(DEV)
    b, sb = pq.fp8_quant(w, block)[:2]
    q, s = pq.fp8_quant(x)[:2]
    want = pq.fp8_gemm(q, s, b, sb, block)
    far = torch.empty(19 * pitch + 512, dtype=torch.bfloat16, device=DEV)
    fx = far.as_strided((rows, cols), (pitch, 1))
    fx.copy_(x)
    codes = torch.empty(19 * pitch + 512, dtype=torch.uint8, device=DEV)
    fq = codes.as_strided((rows, cols), (pitch, 1))
    fs = torch.empty_like(s)
    pq.pq_fp8_quant(R.ROW, fx, fq, fs)
    assert torch.equal(fq, q.view(torch.uint8)) and torch.equal(fs, s)
    fy = far.as_strided((rows, 50), (pitch, 1))
    pq.pq_fp8_gemm(fq, fs, b, sb, block, fy)
    assert torch.equal(fy, want)
    pq.pq_fp8_gemm(fq, fs, b, sb, block, far[8:].as_strided((rows, 50), (pitch - 8, 1)))
    assert torch.equal(far[8:].as_strided((rows, 50), (pitch - 8, 1)), want)


@pytest.mark.parametrize("block", [R.TILE, R.ROW])
def test_quantization_of_more_than_2_31_values(pq, block):  # noqa: F811
    rows, cols = (1 << 20) + 128 * 37 + 3, 2040
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = draw(131, cols, 3, torch.bfloat16)
    first = rows // 128 * 128 - 128  # a tile's border
    x[first:] = tail.to(DEV)
    q, s, qt, st = pq.fp8_quant(x, block, transposed=True)
    want, ws = R.quant(tail, block)
    same_codes(q[first:], want)
    assert torch.equal((s[:, first:] if block == R.ROW else s[first // 128:]).cpu(), ws)
    want, ws = R.quant(tail.t().contiguous(), block)
    same_codes(qt[:, first:].contiguous(), want)
    assert torch.equal((st[first // 128:] if block == R.ROW else st[:, first // 128:]).cpu(), ws)
    assert not q[:first].view(torch.uint8).any() and not qt[:, :first].view(torch.uint8).any()


def test_clipping_of_more_than_2_31_values(pq):  # noqa: F811
    n = (1 << 31) + 77
    t = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t[5], t[1 << 31], t[-1], t[-40] = 3.0, -4.0, 12.0, 84.0
    norm, coef = outs()
    pq.pq_grad_clip(pq.tensor_array([t]), 10.0, norm, coef, scratch(pq, 1))
    want = math.sqrt(9 + 16 + 144 + 84 * 84)
    assert float(norm) == pytest.approx(want, rel=RTOL)
    assert float(coef) == pytest.approx(coef_of(want, 10.0), rel=RTOL)
    at = torch.tensor([5, 1 << 31, n - 1, n - 40], device=DEV)
    assert torch.equal(t[at], (torch.tensor([3.0, -4.0, 12.0, 84.0], device=DEV) * coef).to(torch.bfloat16))
    assert int(torch.count_nonzero(t)) == 4
