"""Block quantization to e4m3 and the block-scaled product on the GPU against
their definitions in 64 bits: codes and scales bit for bit, products within a
bound counted in roundings."""
import pytest
import torch

from tests import fp8_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_b200 import pq
    return pq


def draw(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x *= torch.where(torch.rand(cols, generator=g) < 0.05, 20.0, 1.0)
    return x.to(dtype)


def same_codes(got, want):
    assert torch.equal(got.float().cpu().double(), want), "codes differ from the definition"


SHAPES = [(1, 1), (1, 127), (1, 4096), (3, 128), (16, 4096), (127, 129), (128, 128), (129, 257),
          (130, 136), (5, 2047), (300, 72), (257, 1024)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("block", [R.ROW, R.TILE])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quant_matches_the_definition(pq, rows, cols, block, dtype):
    x = draw(rows, cols, rows * 7 + cols, DTYPES[dtype])
    q, s, qt, st = pq.fp8_quant(x.to(DEV), block, transposed=True)
    for got, gs, v in ((q, s, x), (qt, st, x.t().contiguous())):
        want, ws = R.quant(v, block)
        same_codes(got, want)
        assert torch.equal(gs.cpu(), ws)
    # each output alone is the same
    for kw in ({}, {"transposed": False}):
        q1, s1, a, b = pq.fp8_quant(x.to(DEV), block, **kw)
        assert a is None and b is None
        same_codes(q1, R.quant(x, block)[0])
        assert torch.equal(s1.cpu(), s.cpu())
    qt2, st2 = pq.fp8_empty(cols, rows, DEV), torch.empty_like(st)
    pq.pq_fp8_quant(block, x.to(DEV), qt_out=qt2, st_out=st2)
    assert torch.equal(qt2.float(), qt.float()) and torch.equal(st2, st)


@pytest.mark.parametrize("block", [R.ROW, R.TILE])
@pytest.mark.parametrize("dx,pitch", [(0, 200), (1, 200), (8, 208), (3, 197)])
def test_quant_strided_input_and_untouched_padding(pq, block, dx, pitch):
    rows, cols = 133, 170
    base = draw(rows, pitch, 5, torch.bfloat16).to(DEV)
    x = base[:, dx:dx + cols]
    out = torch.full((rows, 192), 0x55, dtype=torch.uint8, device=DEV)
    out_t = torch.full((cols, 144), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.empty(pq.fp8_scale_shape(block, rows, cols), device=DEV)
    st = torch.empty(pq.fp8_scale_shape(block, cols, rows), device=DEV)
    pq.pq_fp8_quant(block, x, out[:, :cols], s, out_t[:, :rows], st)
    same_codes(out[:, :cols].view(torch.float8_e4m3fn), R.quant(x.cpu(), block)[0])
    same_codes(out_t[:, :rows].view(torch.float8_e4m3fn), R.quant(x.t().cpu().contiguous(), block)[0])
    assert (out[:, cols:] == 0x55).all() and (out_t[:, rows:] == 0x55).all()


def test_quant_odd_output_pitch_takes_element_stores(pq):
    x = draw(40, 150, 6, torch.float32).to(DEV)
    out = torch.zeros((40, 151), dtype=torch.uint8, device=DEV)
    s = torch.empty(pq.fp8_scale_shape(R.ROW, 40, 150), device=DEV)
    pq.pq_fp8_quant(R.ROW, x, out[:, 1:], s)
    same_codes(out[:, 1:].contiguous().view(torch.float8_e4m3fn), R.quant(x.cpu(), R.ROW)[0])
    assert (out[:, 0] == 0).all()


def test_quant_extreme_values(pq):
    x = torch.zeros(8, 256)
    x[1, :128] = 1e-40                       # below the smallest maximum a scale is made from
    x[2, 3], x[2, 4] = 3e38, -1.0            # the largest magnitudes
    x[3] = torch.linspace(-448, 448, 256)    # ties and the largest code
    x[3, 0] = 448.0
    x[4, 7] = 2.0 ** -96
    x[5, :] = -0.0
    want, ws = R.quant(x, R.ROW)
    q, s, qt, st = pq.fp8_quant(x.to(DEV), R.ROW, transposed=True)
    same_codes(q, want)
    assert torch.equal(s.cpu(), ws) and torch.isfinite(s).all()
    same_codes(qt, R.quant(x.t().contiguous(), R.ROW)[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("block", [R.ROW, R.TILE])
def test_nan_and_inf_reach_the_product(pq, bad, block):
    x = draw(130, 300, 8)
    x[5, 140] = bad
    q, s, _, _ = pq.fp8_quant(x.to(DEV), R.ROW)
    b, sb, _, _ = pq.fp8_quant(draw(20, 300, 9).to(DEV), block)
    assert not torch.isfinite(s[1, 5]) and torch.isfinite(s[0]).all() and torch.isfinite(s[2]).all()
    y = pq.fp8_gemm(q, s, b, sb, block)
    assert torch.isnan(y[5]).all()
    assert torch.isfinite(y[:5]).all() and torch.isfinite(y[6:]).all()
    # in B, they reach that column (and with tiles the columns that share its scale)
    w, sw, _, _ = pq.fp8_quant(x.to(DEV), block)
    y = pq.fp8_gemm(b, pq.fp8_quant(draw(20, 300, 9).to(DEV), R.ROW)[1], w, sw, block)
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, 128:]).all()


def check_product(pq, m, n, k, block, out, seed=0, std=1.0):
    a, sa, _, _ = pq.fp8_quant(draw(m, k, seed + 1).to(DEV), R.ROW)
    b, sb, _, _ = pq.fp8_quant(draw(n, k, seed + 2, std=std).to(DEV), block)
    y = pq.fp8_gemm(a, sa, b, sb, block, out_dtype=DTYPES[out])
    assert y.shape == (m, n) and y.dtype == DTYPES[out]
    want, mags = R.product(a, sa, b, sb, block)
    err = (y.cpu().double() - want).abs()
    tol = R.product_tolerance(want, mags, k, DTYPES[out])
    assert (err <= tol).all(), f"off by {float((err / tol).max())} tolerances"
    assert pq.pq_device_status() == pq.PQ_OK
    return a, sa, b, sb, y


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 130, 257), (7, 64, 8192), (16, 1024, 4096),
            (77, 1000, 1536), (128, 128, 128), (129, 127, 130), (130, 256, 384), (255, 513, 1000),
            (300, 2048, 640), (512, 512, 4111), (1000, 5632, 2048), (64, 14336, 512),
            (2048, 2050, 384), (1990, 4099, 200), (2300, 2048, 100)]


@pytest.mark.parametrize("block", [R.TILE, R.ROW])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product_matches_64_bits(pq, m, n, k, block):
    check_product(pq, m, n, k, block, "bf16", seed=m + n + k)


@pytest.mark.parametrize("out", ["fp32", "fp16"])
@pytest.mark.parametrize("block", [R.TILE, R.ROW])
@pytest.mark.parametrize("m,n,k", [(1, 300, 700), (33, 129, 128), (260, 390, 1290), (1100, 2056, 520), (2000, 2047, 260)])
def test_product_output_types(pq, m, n, k, block, out):
    check_product(pq, m, n, k, block, out, seed=m, std=0.05)


def test_product_is_deterministic(pq):
    a, sa, b, sb, y = check_product(pq, 9, 640, 4096, R.TILE, "fp32")
    for _ in range(5):
        assert torch.equal(pq.fp8_gemm(a, sa, b, sb, R.TILE, out_dtype=torch.float32), y)


def test_product_writes_only_its_rows(pq):
    a, sa, b, sb, y = check_product(pq, 40, 72, 256, R.TILE, "bf16")
    for pad in (8, 5):  # aligned and odd pitches
        big = torch.full((42, 72 + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        pq.pq_fp8_gemm(a, sa, b, sb, R.TILE, big[1:41, :72])
        assert torch.equal(big[1:41, :72], y)
        assert (big[0] == 7).all() and (big[41] == 7).all() and (big[:, 72:] == 7).all()


def test_product_of_views(pq):
    """Codes with a wider pitch than their rows, uint8 codes, a single row of
    any pitch."""
    a, sa, b, sb, y = check_product(pq, 40, 72, 256, R.TILE, "bf16")
    wide = torch.zeros((40, 512), dtype=torch.uint8, device=DEV)
    wide[:, 128:384] = a.view(torch.uint8)
    assert torch.equal(pq.fp8_gemm(wide[:, 128:384], sa, b, sb, R.TILE), y)
    one = a[:1].view(torch.uint8).clone()[:, :250]
    one = torch.cat([one.flatten(), one.flatten()]).view(2, 250)[:1]  # pitch 250
    y1 = pq.fp8_gemm(one, sa[:, :1].contiguous(), b[:, :250], sb, R.TILE)
    y2 = pq.fp8_gemm(a[:1, :250], sa[:, :1].contiguous(), b[:, :250], sb, R.TILE)
    assert torch.equal(y1, y2)


def test_empty_products(pq):
    e = lambda r, c: pq.fp8_empty(r, c, DEV)
    f = lambda *s: torch.empty(s, device=DEV)
    n0 = pq.pq_launch_count()
    assert pq.fp8_gemm(e(0, 64), f(1, 0), e(5, 64), f(1, 1), R.TILE).shape == (0, 5)
    assert pq.fp8_gemm(e(5, 64), f(1, 5), e(0, 64), f(0, 1), R.TILE).shape == (5, 0)
    assert pq.fp8_quant(torch.empty(0, 5, device=DEV), R.ROW, transposed=True)[0].shape == (0, 5)
    assert pq.pq_launch_count() == n0
    y = pq.fp8_gemm(e(5, 0), f(0, 5), e(6, 0), f(0, 6), R.ROW, out_dtype=torch.float32)
    assert torch.equal(y.cpu(), torch.zeros(5, 6))


def test_another_stream_and_graph_replay(pq):
    x = draw(50, 700, 3, torch.bfloat16).to(DEV)
    w = draw(300, 700, 4, torch.bfloat16).to(DEV)
    b, sb, _, _ = pq.fp8_quant(w, R.TILE)
    q, s, _, _ = pq.fp8_quant(x, R.ROW)
    want = pq.fp8_gemm(q, s, b, sb)
    y = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pq.pq_fp8_gemm(q, s, b, sb, R.TILE, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    q2, s2, y2 = pq.fp8_empty(50, 700, DEV), torch.zeros_like(s), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.pq_fp8_quant(R.ROW, x, q2, s2)
        pq.pq_fp8_gemm(q2, s2, b, sb, R.TILE, y2)
    for scale in (1.0, 4.0):
        x.mul_(scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, want * scale)  # a power of two moves the scales alone
    x.mul_(0.25)


def test_two_streams_at_once(pq):
    """Calls share no state: products and quantizations that overlap on the
    GPU give what they give alone."""
    sets = []
    for i, (m, n, k, block) in enumerate([(700, 1500, 1100, R.TILE), (5, 640, 3000, R.ROW), (2000, 2050, 300, R.ROW)]):
        x, w = draw(m, k, i, torch.bfloat16).to(DEV), draw(n, k, i + 9, torch.bfloat16).to(DEV)
        b, sb, _, _ = pq.fp8_quant(w, block)
        q, s, _, _ = pq.fp8_quant(x, R.ROW)
        sets.append((x, q, s, b, sb, block, pq.fp8_gemm(q, s, b, sb, block)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[] for _ in sets]
    for _ in range(8):
        for st, (x, q, s, b, sb, block, _), o in zip(streams, sets, outs):
            with torch.cuda.stream(st):
                q2, s2, _, _ = pq.fp8_quant(x, R.ROW)
                o.append(pq.fp8_gemm(q2, s2, b, sb, block))
    torch.cuda.synchronize()
    for o, (*_, want) in zip(outs, sets):
        assert all(torch.equal(y, want) for y in o)


def test_waits_give_up_with_a_status(pq):
    for m, n, k, block in ((40, 300, 1024, R.ROW), (33, 4096, 520, R.TILE), (1100, 2056, 520, R.TILE),
                           (1100, 2056, 520, R.ROW)):
        a, sa, b, sb, y = check_product(pq, m, n, k, block, "bf16")
        pq.pq_debug_abort_waits(True)
        try:
            pq.fp8_gemm(a, sa, b, sb, block)
            assert pq.pq_device_status() == pq.PQ_ERR_TIMEOUT
        finally:
            pq.pq_debug_abort_waits(False)
        assert pq.pq_device_status() == pq.PQ_OK
        assert torch.equal(pq.fp8_gemm(a, sa, b, sb, block), y)


# --------------------------------------------------------- the linear layer
def linear_reference(x, w, dy):
    """The three products in 64 bits from the quantized operands."""
    v = lambda t, block: R.values(*(lambda q, s: (q.to(torch.float32).to(torch.float8_e4m3fn), s))(*R.quant(t, block)), block)
    xr, xc = v(x, R.ROW), v(x.t().contiguous(), R.ROW)
    yr, yc = v(dy, R.ROW), v(dy.t().contiguous(), R.ROW)
    wt = v(w, R.TILE)
    return {"y": (xr @ wt.t(), xr.abs() @ wt.abs().t(), x.shape[1]),
            "dx": (yr @ wt, yr.abs() @ wt.abs(), dy.shape[1]),
            "dw": (yc @ xc.t(), yc.abs() @ xc.abs().t(), x.shape[0])}


@pytest.mark.parametrize("m,n,k", [(1, 128, 256), (37, 200, 130), (129, 384, 520), (300, 257, 1024)])
def test_linear_step(pq, m, n, k):
    from bit_quantization_aware_b200.linear import Fp8Linear
    x, w, dy = (draw(r, c, r + c, torch.bfloat16, std) for r, c, std in ((m, k, 1.0), (n, k, 0.05), (m, n, 1e-3)))
    layer = Fp8Linear(n, k, m + 40, device=DEV)  # more room than tokens
    y = layer.forward(x.to(DEV), w.to(DEV))
    dx, dw = layer.backward(dy.to(DEV))
    ref = linear_reference(x, w, dy)
    for name, got in (("y", y), ("dx", dx), ("dw", dw)):
        want, mags, kk = ref[name]
        tol = R.product_tolerance(want, mags, kk, torch.bfloat16)
        assert ((got.cpu().double() - want).abs() <= tol).all(), name


def test_linear_gradients_against_differences(pq):
    """Along directions that keep every block's maximum (the elements that are
    not maxima move by whole steps of their codes), the loss sum(y * dy) moves
    by <dx, u>: with power-of-two scales nothing is rounded away."""
    from bit_quantization_aware_b200.linear import Fp8Linear
    m, n, k = 24, 40, 160
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-4, 5, (m, k), generator=g).float()
    w = torch.randint(-4, 5, (n, k), generator=g).float()
    dy = torch.randint(-4, 5, (m, n), generator=g).float()
    for t in (x, w, dy):  # the same maximum in every block: scales 7/448 = 2^-6
        t[:, ::16], t[::8, :] = 7.0, 7.0
    layer = Fp8Linear(n, k, m, device=DEV)
    run = lambda a, b: layer.forward(a.to(DEV), b.to(DEV), torch.empty(m, n, device=DEV)).cpu().double()
    y0 = run(x, w)
    assert torch.equal(y0, x.double() @ w.double().t())
    dx, dw = layer.backward(dy.to(DEV), torch.empty(m, k, device=DEV), torch.empty(n, k, device=DEV))
    ux, uw = (torch.where(t.abs() < 6, torch.randint(-1, 2, t.shape, generator=g).float(), 0.0) for t in (x, w))
    loss = lambda y: float((y * dy.double()).sum())
    assert loss(run(x + ux, w)) - loss(y0) == float((dx.cpu().double() * ux.double()).sum())
    assert loss(run(x, w + uw)) - loss(y0) == float((dw.cpu().double() * uw.double()).sum())


@pytest.mark.parametrize("as_int", [False, True])
def test_outputs_belong_to_the_stream_that_writes_them(pq, as_int):
    """Memory that the current stream's pool holds free may still be in use
    there: a call on another stream takes none of it."""
    from bit_quantization_aware_b200.linear import Fp8Linear
    m, n, k = 700, 640, 512
    x, w = (draw(r, k, r, torch.bfloat16).to(DEV) for r in (m, n))
    dy = draw(m, n, 1, torch.bfloat16).to(DEV)
    layer = Fp8Linear(n, k, m, device=DEV)
    want = [pq.fp8_gemm(*pq.fp8_quant(x)[:2], *pq.fp8_quant(w, 2)[:2])]
    want += [layer.forward(x, w), *layer.backward(dy)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    # every size that the calls allocate, free in the current stream's pool
    free = [torch.empty(b, dtype=torch.uint8, device=DEV)
            for b in (m * k, n * k, 4 * 4 * m, 4 * 5 * 4, 2 * m * n, 2 * m * k, 2 * n * k) for _ in range(4)]
    held = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in free]
    del free
    q = pq.fp8_quant(x, stream=stream)
    b = pq.fp8_quant(w, 2, stream=stream)
    y = pq.fp8_gemm(*q[:2], *b[:2], stream=stream)
    got = [y, layer.forward(x, w, stream=stream), *layer.backward(dy, stream=stream)]
    side.synchronize()
    for t in (*q[:2], *b[:2], *got):
        assert not any(lo <= t.data_ptr() < hi for lo, hi in held)
    for a, e in zip(got, want):
        assert torch.equal(a, e)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_one_row_of_any_pitch(pq, out):
    """One row has no pitch to speak of: a number that no TMA map takes is
    no reason to refuse it."""
    n, k = 4000, 128  # one K block: not split
    a, b = pq.fp8_quant(draw(1, k, 1).to(DEV))[:2], pq.fp8_quant(draw(n, k, 2).to(DEV), 2)[:2]
    want = pq.fp8_gemm(*a, *b, out_dtype=out)
    y = torch.empty(n, dtype=out, device=DEV).as_strided((1, n), (1 << 41, 1))
    pq.pq_fp8_gemm(*a, *b, pq.PQ_BLOCK_TILE, y)
    assert torch.equal(y[0], want[0])
