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


# every kernel that the sizes can choose: (columns of a tile, CTAs of a tile's K split)
KERNELS = [(R.TILE, w, s) for w in (64, 128) for s in (1, 2, 4, 8)] + [(R.TILE, 256, 1)] + \
    [(R.ROW, 64, s) for s in (1, 2, 4, 8)] + [(R.ROW, 256, 1)]


@pytest.fixture()
def force(pq):  # noqa: F811
    yield pq.pq_debug_fp8_force
    pq.pq_debug_fp8_force(0, 0)


def kernel_shapes(split):
    """Ragged everywhere; one row; rows and columns beside a tile's border; K
    blocks that CTAs share unevenly, and one each."""
    return [(1, 1867, 3167), (46, 333, 1926), (129, 130, 1024), (300, 257, 1153), (257, 515, 128 * split),
            (128, 64, 128 * split + 1), (2, 1, 1100)]


@pytest.mark.parametrize("block,width,split", KERNELS)
def test_every_kernel(pq, force, block, width, split):  # noqa: F811
    force(width, split)
    for i, (m, n, k) in enumerate(kernel_shapes(split)):
        assert pq.pq_debug_fp8_choice(m, n, k, block) == (width, split)
        out = ("bf16", "fp16", "fp32")[(i + width + split) % 3]
        check_product(pq, m, n, k, block, out, seed=7 * i + split, std=0.05)


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block,width,split", KERNELS)
def test_every_kernel_writes_its_rows_alone(pq, force, block, width, split, out):  # noqa: F811
    """Every output type, aligned and odd pitches, with what lies around y."""
    force(width, split)
    m, n, k = 133, 198, 1030
    a, sa, b, sb, want = check_product(pq, m, n, k, block, out, seed=width + split, std=0.05)
    for pad in (2, 3, 58):  # 200: 8-byte or 16-byte rows, 201: odd, 256
        big = torch.full((m + 2, n + pad), 7.0, dtype=want.dtype, device=DEV)
        pq.pq_fp8_gemm(a, sa, b, sb, block, big[1:m + 1, :n])
        assert torch.equal(big[1:m + 1, :n], want)
        assert (big[0] == 7).all() and (big[m + 1] == 7).all() and (big[:, n:] == 7).all()
    assert torch.equal(pq.fp8_gemm(a, sa, b, sb, block, out_dtype=want.dtype), want)


@pytest.mark.parametrize("block,width,split", KERNELS)
def test_waits_of_every_kernel_give_up(pq, force, block, width, split):  # noqa: F811
    force(width, split)
    a, sa, b, sb, y = check_product(pq, 600, 700, 2100, block, "bf16")
    pq.pq_debug_abort_waits(True)
    try:
        pq.fp8_gemm(a, sa, b, sb, block)
        assert pq.pq_device_status() == pq.PQ_ERR_TIMEOUT
    finally:
        pq.pq_debug_abort_waits(False)
    assert pq.pq_device_status() == pq.PQ_OK
    assert torch.equal(pq.fp8_gemm(a, sa, b, sb, block), y)


def test_the_sizes_choose_every_kernel(pq):  # noqa: F811
    """No kernel is there for nothing: sizes of decode batches to training
    batches reach each one."""
    g = torch.Generator().manual_seed(0)
    log = lambda lo, hi, n: torch.exp(torch.rand(n, generator=g) * (hi / lo).log() + lo.log()).long().tolist()
    t = lambda v: torch.tensor(float(v))
    sizes = zip(log(t(1), t(8192), 20000), log(t(64), t(14336), 20000), log(t(64), t(14336), 20000))
    seen = {(block, *pq.pq_debug_fp8_choice(m, n, k, block)) for m, n, k in sizes for block in (R.TILE, R.ROW)}
    assert seen == set(KERNELS)


def test_a_product_that_a_forced_kernel_cannot_take(pq, force):  # noqa: F811
    a, b = pq.fp8_quant(draw(5, 300, 1).to(DEV))[:2], pq.fp8_quant(draw(6, 300, 2).to(DEV))[:2]
    want = pq.fp8_gemm(*a, *b, R.ROW)
    for width, split in ((128, 1), (64, 4)):  # no such kernel; three K blocks
        force(width, split)
        with pytest.raises(pq.PQError):
            pq.fp8_gemm(*a, *b, R.ROW)
    force(0, 0)
    assert torch.equal(pq.fp8_gemm(*a, *b, R.ROW), want)
