"""The kernels of the block-scaled product one by one."""
import pytest
import torch

from tests import fp8_ref as R
from tests.test_fp8_gpu import DEV, check_product, draw, pq  # noqa: F401 (pq is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [R.TILE, R.ROW])
def test_pairs_beside_other_traffic(pq, block):  # noqa: F811
    """The issuing CTA of a pair waits for both CTAs' copies itself: however
    late the other's arrive, because other streams keep memory busy, the sums
    are those of a quiet GPU."""
    m, n, k = 2048, 2560, 2000
    a, sa, b, sb, want = check_product(pq, m, n, k, block, "fp32", seed=3)
    busy = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    codes = pq.fp8_quant(draw(4096, 4096, 5, torch.bfloat16).to(DEV))
    outs = [torch.empty_like(want) for _ in range(24)]
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(12):
            busy.add_(1)
    with torch.cuda.stream(other):
        for _ in range(6):
            pq.fp8_gemm(*codes[:2], *codes[:2], R.ROW)
    for y in outs:
        pq.pq_fp8_gemm(a, sa, b, sb, block, y)
    torch.cuda.synchronize()
    assert pq.pq_device_status() == pq.PQ_OK
    assert all(torch.equal(y, want) for y in outs)
