"""Ends of the block-scaled product's operands that fall inside 16 bytes: what
lies beside Y stays, and what lies beside A and B is not read."""
import pytest
import torch

from tests import fp8_ref as R
from tests.test_fp8_gpu import DEV, DTYPES, check_product, draw, pq  # noqa: F401 (pq is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("block", [R.TILE, R.ROW])
@pytest.mark.parametrize("m,n,k", [(133, 198, 130), (700, 2049, 260), (2300, 4100, 140), (3000, 2302, 384)])
def test_columns_beside_y_stay(pq, m, n, k, block, out):  # noqa: F811
    """A pitch and a base that suit wide stores, and a last column that does
    not end one."""
    a, sa, b, sb, want = check_product(pq, m, n, k, block, out, seed=n)
    pitch = (n + 7) // 8 * 8
    for pad in (0, 8):
        big = torch.full((m + 1, pitch + pad), 7.0, dtype=want.dtype, device=DEV)
        pq.pq_fp8_gemm(a, sa, b, sb, block, big[:m, :n])
        assert torch.equal(big[:m, :n], want)
        assert (big[:, n:] == 7).all() and (big[m] == 7).all()


def test_memory_behind_one_row_stays(pq):  # noqa: F811
    """One row of 4001 with a pitch of 4008: the row's end is the tensor's."""
    a, sa, b, sb, want = check_product(pq, 1, 4001, 100, R.TILE, "bf16")
    flat = torch.full((4008,), 7.0, dtype=torch.bfloat16, device=DEV)
    pq.pq_fp8_gemm(a, sa, b, sb, R.TILE, flat.as_strided((1, 4001), (4008, 1)))
    assert torch.equal(flat[:4001], want[0]) and (flat[4001:] == 7).all()


@pytest.mark.parametrize("block", [R.TILE, R.ROW])
@pytest.mark.parametrize("m,n,k", [(1, 130, 1), (9, 300, 1030), (140, 200, 127), (2000, 2050, 265)])
def test_codes_beside_a_and_b_are_not_read(pq, m, n, k, block):  # noqa: F811
    """The pitch's bytes behind k hold NaN codes."""
    a, sa, b, sb, want = check_product(pq, m, n, k, block, "fp32", seed=k)
    pitch = (k + 15) // 16 * 16 + 16
    wide = []
    for q in (a, b):
        w = torch.full((q.shape[0], pitch), 0x7F, dtype=torch.uint8, device=DEV)
        w[:, :k] = q.view(torch.uint8)
        wide.append(w[:, :k])
    assert torch.equal(pq.fp8_gemm(wide[0], sa, wide[1], sb, block, out_dtype=torch.float32), want)
