"""The global gradient norm, clipping and the clipped quantizer updates on
the GPU against 64-bit references."""
import math

import numpy as np
import pytest
import torch

from bit_quantization_aware_b200 import inputs as I

pytestmark = pytest.mark.gpu

DEV = "cuda"
# fp64 squares and sums are off by a few 2^-53 times the number of terms, far
# below the one rounding of the result to fp32 (2^-24 relative); twice that
# covers it and the reference's own rounding
RTOL = 2.0 ** -23
QS = ["binary", "ternary", "seq2", "seq2_b", "lsq2", "lsq3", "lsq4"]


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_b200 import pq
    return pq


def scratch(pq, n, mats=0):
    # any contents
    return torch.full((pq.pq_grad_norm_workspace_bytes(n, mats),), 0xFF, dtype=torch.uint8, device=DEV)


def outs():
    return [torch.full((1,), 7.0, device=DEV) for _ in range(2)]


def coef_of(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))


def make(n, dtype, seed, offset=0, std=1e-3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(n + offset, device=DEV, generator=g) * std).to(dtype)[offset:]


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


SETS = {
    "one element": [(1, torch.float32, 0)],
    "empty among others": [(0, torch.bfloat16, 0), (5, torch.bfloat16, 0), (0, torch.float32, 0)],
    "unit borders": [(8191, torch.float32, 0), (8192, torch.float32, 0), (8193, torch.float32, 0),
                     (16384, torch.bfloat16, 0), (16385, torch.float16, 0)],
    "odd offsets": [(1000, torch.float32, 1), (1000, torch.bfloat16, 1), (70001, torch.float16, 3)],
    "all types": [(300000, torch.bfloat16, 0), (123457, torch.float32, 0), (99999, torch.float16, 0)],
    "many": [(i * 37 % 911 + 1, torch.float32, 0) for i in range(600)],
    "large": [(5_000_003, torch.bfloat16, 0), (3_000_001, torch.float32, 0)],
}


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("max_norm", [0.01, 1e9])
def test_norm_and_clip(pq, name, max_norm):
    ts = [make(n, d, i, off) for i, (n, d, off) in enumerate(SETS[name])]
    want = norm64(ts)
    norm, coef = outs()
    sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
    pq.pq_grad_norm(max_norm, norm, coef, scratch(pq, len(ts)), tensors=pq.tensor_array(ts), sumsq_out=sumsq)
    assert float(norm) == pytest.approx(want, rel=RTOL)
    assert float(sumsq) == pytest.approx(want * want, rel=1e-12)
    assert float(coef) == pytest.approx(coef_of(want, max_norm), rel=RTOL)
    keep = [t.clone() for t in ts]
    n2, c2 = outs()
    # out of place, in fp32 (one fp32 product, no further rounding) ...
    big = [torch.full_like(t, 3.0, dtype=torch.float32) for t in ts]
    pq.pq_grad_clip(pq.tensor_array(ts, big), max_norm, n2, c2, scratch(pq, len(ts)))
    assert torch.equal(n2, norm) and torch.equal(c2, coef)
    for t, k, b in zip(ts, keep, big):
        assert torch.equal(t, k) and torch.equal(b, k.float() * coef)
    # ... and in place, in the tensor's own type
    pq.pq_grad_clip(pq.tensor_array(ts), max_norm, n2, None, scratch(pq, len(ts)))
    assert torch.equal(n2, norm)
    for t, k in zip(ts, keep):
        assert torch.equal(t, (k.float() * coef).to(k.dtype))


def test_in_place_matches_and_leaves_neighbours(pq):
    flat = make(10_000, torch.bfloat16, 3)
    keep = flat.clone()
    parts = [flat[10:500], flat[501:3000], flat[4096:9000]]
    norm = pq.clip_grad_norm(parts, 1e-3)
    want = norm64([keep[10:500], keep[501:3000], keep[4096:9000]])
    assert float(norm) == pytest.approx(want, rel=RTOL)
    c = torch.tensor([coef_of(want, 1e-3)], dtype=torch.float64, device=DEV).float()
    for a, b in ((10, 500), (501, 3000), (4096, 9000)):
        # coef itself is within one fp32 rounding: products agree to a bf16 step
        assert torch.allclose(flat[a:b].float(), keep[a:b].float() * c, rtol=2 ** -8 + 2 ** -22, atol=0)
    for a, b in ((0, 10), (500, 501), (3000, 4096), (9000, 10_000)):
        assert torch.equal(flat[a:b], keep[a:b])


@pytest.mark.parametrize("value", [1e-25, 3e30, 2.0 ** -133])
def test_range_of_squares(pq, value):
    """Squares that fp32 cannot hold."""
    t = torch.full((4097,), value, dtype=torch.bfloat16, device=DEV)
    norm, coef = outs()
    pq.pq_grad_norm(1.0, norm, coef, scratch(pq, 1), tensors=pq.tensor_array([t]))
    want = math.sqrt(4097) * float(t[0])
    # a norm below 2^-126 rounds to a multiple of 2^-149
    assert float(norm) == pytest.approx(want, rel=RTOL, abs=2.0 ** -150)
    assert float(coef) == pytest.approx(coef_of(want, 1.0), rel=RTOL)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_inf_and_nan(pq, bad):
    ts = [make(5000, torch.float32, 1), make(300, torch.bfloat16, 2)]
    ts[0][4321] = bad
    norm, coef = outs()
    pq.pq_grad_clip(pq.tensor_array(ts), 1.0, norm, coef, scratch(pq, 2))
    if math.isinf(bad):
        assert float(norm) == math.inf and float(coef) == 0.0
        assert torch.isnan(ts[0][4321]) and int(torch.isnan(ts[0]).sum()) == 1 and (ts[1] == 0).all()
    else:
        assert math.isnan(float(norm)) and math.isnan(float(coef))
        assert torch.isnan(ts[0]).all() and torch.isnan(ts[1]).all()


def test_no_gradients(pq):
    norm, coef = outs()
    pq.pq_grad_norm(1.0, norm, coef, scratch(pq, 0))
    assert float(norm) == 0 and float(coef) == 1
    t = torch.zeros(0, device=DEV)
    norm, coef = outs()
    pq.pq_grad_clip(pq.tensor_array([t]), 0.0, norm, coef, scratch(pq, 1))
    assert float(norm) == 0 and float(coef) == 0  # max_norm 0


def test_scale_by_one_writes_nothing_and_by_two(pq):
    t = make(30_000, torch.float32, 5)
    t[7] = float("nan")  # a product by 1 would keep it; the bits stay too
    keep = t.clone()
    one = torch.ones(1, device=DEV)
    pq.pq_grad_scale(pq.tensor_array([t]), one)
    assert torch.equal(t.view(torch.int32), keep.view(torch.int32))
    o = torch.zeros_like(t)
    pq.pq_grad_scale(pq.tensor_array([t], [o]), one)
    assert torch.equal(o[8:], keep[8:]) and torch.isnan(o[7])
    pq.pq_grad_scale(pq.tensor_array([t]), 2 * one)
    assert torch.equal(t[8:], 2 * keep[8:])


def test_deterministic_and_in_a_graph(pq):
    ts = [make(700_001, torch.bfloat16, 1), make(65_537, torch.float32, 2)]
    arr, ws = pq.tensor_array(ts), scratch(pq, 2)
    big = [torch.empty_like(t, dtype=torch.float32) for t in ts]
    arr_out = pq.tensor_array(ts, big)
    norm, coef = outs()
    pq.pq_grad_norm(0.1, norm, coef, ws, tensors=arr)
    for _ in range(4):
        n, c = outs()
        pq.pq_grad_norm(0.1, n, c, ws, tensors=arr)
        assert torch.equal(n, norm) and torch.equal(c, coef)
    n, c = outs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.pq_grad_clip(arr_out, 0.1, n, c, ws)
    for scale in (1.0, 3.0):
        for t in ts:
            t.mul_(scale)
        g.replay()
        torch.cuda.synchronize()
        assert float(n) == pytest.approx(norm64(ts), rel=RTOL)
        for t, b in zip(ts, big):
            assert torch.equal(b, t.float() * c)


def test_a_stream_of_its_own_sees_earlier_work(pq):
    side = torch.cuda.Stream()
    t = torch.zeros(3_000_000, device=DEV)
    torch.cuda.synchronize()
    norm, coef = outs()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(20):
            t.fill_(float(i))
            pq.pq_grad_clip(pq.tensor_array([t]), 1.0, norm, coef, scratch(pq, 1))
            # the clipped tensor's norm, from the next call on the stream
            n2, c2 = outs()
            pq.pq_grad_norm(1e9, n2, c2, scratch(pq, 1), tensors=pq.tensor_array([t]))
    side.synchronize()
    want = 19 * math.sqrt(3_000_000)
    assert float(norm) == pytest.approx(want, rel=RTOL)
    assert float(n2) == pytest.approx(want * coef_of(want, 1.0), rel=4 * RTOL)


# --------------------------------------------------- the quantizer's gradient
def matrices(pq, shapes, qname, seed=0, misalign=False):
    q = pq.QUANTIZERS[qname]
    ms = []
    for i, (r, c) in enumerate(shapes):
        w = I.normal_weights(r, c, seed=seed, stream=i)
        a = I.alpha_init(w, q)
        if qname in ("seq2", "ternary"):
            a = a * 0.7  # some weights outside the clip range
        g = I.grad_bf16(r, c, seed=seed, stream=i + 64)
        off = 1 if misalign else 0
        dev = lambda t: torch.cat([torch.zeros(off, dtype=t.dtype), t.flatten()]).to(DEV)[off:].view(t.shape)
        ms.append(dict(rows=r, cols=c, w=dev(w), alpha=a.to(DEV), g=dev(g),
                       grad_scale=pq.pq_default_grad_scale(q, c)))
    return q, ms


def backward(pq, q, ms):
    out = [pq.fakequant_bwd(q, m["w"], m["alpha"], m["g"], m["grad_scale"]) for m in ms]
    return [t for pair in out for t in pair]


@pytest.mark.parametrize("qname", QS)
@pytest.mark.parametrize("misalign", [False, True])
def test_quantizer_norm_is_that_of_the_backward(pq, qname, misalign):
    shapes = [(5, 64), (1, 8), (300, 257), (64, 4096), (3, 14336), (7, 1)]
    q, ms = matrices(pq, shapes, qname, misalign=misalign)
    grads = backward(pq, q, ms)
    extra = [make(1001, torch.float32, 4)]
    for m in ms[::2]:
        m["dalpha"] = torch.full((m["rows"],), 9.0, device=DEV)
    norm, coef = outs()
    pq.pq_grad_norm(0.02, norm, coef, scratch(pq, 1, len(ms)), tensors=pq.tensor_array(extra), q=q,
                    mats=pq.matrix_array(ms))
    want = norm64(grads + extra)
    assert float(norm) == pytest.approx(want, rel=RTOL)
    assert float(coef) == pytest.approx(coef_of(want, 0.02), rel=RTOL)
    for i, m in enumerate(ms):
        if "dalpha" in m:
            assert torch.equal(m["dalpha"], grads[2 * i + 1])


def test_quantizer_norm_of_many_and_empty_matrices(pq):
    shapes = [(i % 9, 8 * (i % 5)) for i in range(300)]
    q, ms = matrices(pq, shapes, "seq2")
    for m in ms:
        m["dalpha"] = torch.full((m["rows"],), 9.0, device=DEV)
    norm, coef = outs()
    pq.pq_grad_norm(1.0, norm, coef, scratch(pq, 0, len(ms)), q=q, mats=pq.matrix_array(ms))
    grads = [t for m in ms if m["rows"] and m["cols"] for t in backward(pq, q, [m])]
    assert float(norm) == pytest.approx(norm64(grads), rel=RTOL)
    assert all((m["dalpha"] == 0).all() for m in ms if m["cols"] == 0)


def test_quantizer_norm_against_differences(pq):
    """d(norm^2)/dg along a direction, by central differences of the norm
    itself: norm^2 is quadratic in g, so the difference quotient is exact up
    to rounding (terms of 2^-24 of norm^2 divided by the step)."""
    q, ms = matrices(pq, [(8, 16)], "lsq3")
    m = ms[0]
    g0 = m["g"].clone()
    u = torch.zeros_like(g0)
    u[3, 5] = 2.0 ** -8
    sq = []
    for sign in (1, -1):
        m["g"] = (g0.float() + sign * u.float())
        m["g"] = m["g"].to(torch.bfloat16)
        s = torch.zeros(1, dtype=torch.float64, device=DEV)
        pq.pq_grad_norm(1.0, None, None, scratch(pq, 0, 1), q=q, mats=pq.matrix_array([m]), sumsq_out=s)
        sq.append(float(s))
    m["g"] = g0
    gp, gm = (g0.float() + u.float()).to(torch.bfloat16), (g0.float() - u.float()).to(torch.bfloat16)
    dw_p, da_p = pq.fakequant_bwd(q, m["w"], m["alpha"], gp, m["grad_scale"])
    dw_m, da_m = pq.fakequant_bwd(q, m["w"], m["alpha"], gm, m["grad_scale"])
    want = sum(float(p.double().square().sum() - n.double().square().sum()) for p, n in ((dw_p, dw_m), (da_p, da_m)))
    assert sq[0] - sq[1] == pytest.approx(want, rel=1e-9, abs=1e-15)


def states(ms, seed=5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for m in ms:
        r, c = m["rows"], m["cols"]
        st = dict(m, w=m["w"].clone(), alpha=m["alpha"].clone(),
                  m_w=torch.randn(r, c, device=DEV, generator=g) * 1e-4,
                  v_w=torch.rand(r, c, device=DEV, generator=g) * 1e-7,
                  m_alpha=torch.randn(r, device=DEV, generator=g) * 1e-4,
                  v_alpha=torch.rand(r, device=DEV, generator=g) * 1e-7,
                  dalpha=torch.zeros(r, device=DEV))
        out.append(st)
    return out


KEYS = ("w", "alpha", "m_w", "v_w", "m_alpha", "v_alpha")


@pytest.mark.parametrize("qname", QS)
def test_clipped_adamw_is_adamw_of_scaled_gradients(pq, qname):
    """With a power of two as the factor, scaling the upstream gradient first
    gives the same bits."""
    q, ms = matrices(pq, [(40, 256), (3, 33), (200, 1024)], qname)
    hp_w, hp_a = pq.adamw(3, 1e-3, weight_decay=0.01), pq.adamw(3, 1e-4)
    a, b = states(ms), states(ms)
    for s in b:
        s["g"] = (s["g"].float() * 0.25).to(torch.bfloat16)
    pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array(a), hp_w, hp_a, coef=torch.tensor([0.25], device=DEV))
    pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array(b), hp_w, hp_a)
    c = states(ms)
    pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array(c), hp_w, hp_a, coef=torch.ones(1, device=DEV))
    d = states(ms)
    pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array(d), hp_w, hp_a)
    for x, y, u, v in zip(a, b, c, d):
        for key in KEYS:
            assert torch.equal(x[key], y[key]), key
            assert torch.equal(u[key], v[key]), key
        assert torch.equal(x["dalpha"], v["dalpha"])  # unclipped


@pytest.mark.parametrize("world", [1, 3])
def test_sharded_norm_and_clipped_update(pq, world):
    """Row shards over `world` replicas: the ranks' sums give the norm of the
    averaged gradient, and the clipped update equals the single-GPU one."""
    from bit_quantization_aware_b200.sharded import row_partition
    q, ms = matrices(pq, [(37, 256), (5, 33)], "seq2")
    gs = [[I.grad_bf16(m["rows"], m["cols"], seed=k, stream=i).to(DEV) for i, m in enumerate(ms)]
          for k in range(world)]
    offs, total = [], 0
    for m in ms:
        offs.append(total)
        total += (m["rows"] * m["cols"] + 63) // 64 * 64
    sources = []
    for k in range(world):
        buf = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
        for o, g in zip(offs, gs[k]):
            buf[o:o + g.numel()] = g.flatten()
        sources.append(buf)
    mult = 1.0 / world
    sums = torch.zeros(world, dtype=torch.float64, device=DEV)
    st = states(ms)
    ranks = []
    for k in range(world):
        descs = []
        for s, o in zip(st, offs):
            b, e = row_partition(s["rows"], world)[k]
            descs.append(dict(rows=e - b, cols=s["cols"], g_offset=o + b * s["cols"], grad_scale=s["grad_scale"],
                              **{key: s[key][b:e] for key in KEYS}, dalpha=s["dalpha"][b:e]))
        ranks.append(pq.shard_array(descs))
        pq.pq_reduce_grad_norm(q, sources, mult, ranks[-1], 1.0, None, None, scratch(pq, 0, len(descs)),
                               sumsq_out=sums[k:k + 1])
    norm, coef = outs()
    pq.pq_clip_coef(sums, 0.02, norm, coef)
    # the averaged gradient in 64 bits through the quantizer's mask
    total64 = 0.0
    for i, m in enumerate(ms):
        g = torch.zeros(m["rows"], m["cols"], device=DEV)
        for k in range(world):
            g += gs[k][i].float()
        g = g * mult
        x = (m["w"] / m["alpha"][:, None])
        inside = x.abs() <= torch.tensor(0.99, device=DEV)
        xc = x.clamp(-0.99, 0.99)
        level = (torch.round(xc * 2 - 0.5) + 0.5) / 2
        da = (g.double() * (level.double() - torch.where(inside, x, 0.0).double())).sum(1) * m["grad_scale"]
        total64 += float(torch.where(inside, g, 0.0).double().square().sum() + da.float().double().square().sum())
    # d(alpha) cancels, so its rounding may move the sum by more than the norm's own
    assert float(norm) == pytest.approx(math.sqrt(total64), rel=4 * RTOL)
    assert float(coef) == pytest.approx(coef_of(math.sqrt(total64), 0.02), rel=4 * RTOL)
    hp_w, hp_a = pq.adamw(3, 1e-3), pq.adamw(3, 1e-4)
    if world == 1:
        one = states(ms)
        for s, g in zip(one, gs[0]):
            s["g"] = g
        pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array(one), hp_w, hp_a, coef=coef)
        pq.pq_reduce_bwd_adamw(q, sources, mult, ranks[0], hp_w, hp_a, coef=coef)
        for x, y in zip(st, one):
            for key in KEYS:
                assert torch.equal(x[key], y[key]), key
    else:
        half = torch.tensor([0.5], device=DEV)
        ref = states(ms)
        ref_ranks = []
        for k in range(world):
            descs = []
            for s, o in zip(ref, offs):
                b, e = row_partition(s["rows"], world)[k]
                descs.append(dict(rows=e - b, cols=s["cols"], g_offset=o + b * s["cols"],
                                  grad_scale=s["grad_scale"], **{key: s[key][b:e] for key in KEYS}))
            ref_ranks.append(pq.shard_array(descs))
        for k in range(world):  # 0.5 commutes with every rounding
            pq.pq_reduce_bwd_adamw(q, sources, mult, ranks[k], hp_w, hp_a, coef=half)
            pq.pq_reduce_bwd_adamw(q, sources, mult * 0.5, ref_ranks[k], hp_w, hp_a)
        for x, y in zip(st, ref):
            for key in KEYS:
                assert torch.equal(x[key], y[key]), key


def test_a_training_step_together(pq):
    """Forward of the quantizer, the three products, the norm of the
    quantizer's gradient with another parameter's, the clipped updates."""
    from bit_quantization_aware_b200.linear import Fp8Linear
    m, n, k = 200, 256, 384
    q, ms = matrices(pq, [(n, k)], "seq2")
    st = states(ms)[0]
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(m, k, device=DEV, generator=g).to(torch.bfloat16)
    dy = (torch.randn(m, n, device=DEV, generator=g) * 1e-3).to(torch.bfloat16)
    other = make(n, torch.float32, 9)
    layer = Fp8Linear(n, k, m, device=DEV)
    wq, _ = pq.fakequant_fwd(q, st["w"], st["alpha"])
    y = layer.forward(x, wq)
    dx, _ = layer.backward(dy, dw_out=st["g"])
    assert torch.isfinite(y).all() and torch.isfinite(dx).all()
    dw, da = pq.fakequant_bwd(q, st["w"], st["alpha"], st["g"], st["grad_scale"])
    want = norm64([dw, da, other])
    norm, coef = outs()
    pq.pq_grad_norm(0.5 * want, norm, coef, scratch(pq, 1, 1), tensors=pq.tensor_array([other]), q=q,
                    mats=pq.matrix_array([st]))
    assert float(norm) == pytest.approx(want, rel=RTOL)
    keep = other.clone()
    pq.pq_grad_scale(pq.tensor_array([other]), coef)
    assert torch.equal(other, keep * coef)
    w0 = st["w"].clone()
    m0 = st["m_w"].clone()
    pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array([st]), pq.adamw(1, 1e-3), pq.adamw(1, 1e-4), coef=coef)
    assert torch.equal(st["m_w"], 0.9 * m0 + np.float32(1 - 0.9) * (dw * coef)) or \
        torch.allclose(st["m_w"], 0.9 * m0 + (1 - 0.9) * (dw * coef), rtol=2 ** -21, atol=1e-12)
    assert not torch.equal(st["w"], w0)


@pytest.mark.parametrize("world", [1, 2])
def test_sharded_step_clips_like_the_unsharded(pq, world):
    from bit_quantization_aware_b200.sharded import LocalPeers, ShardedQuantStep
    mats = [I.Matrix("a", 300, 256, 0, 0), I.Matrix("b", 7, 40, 0, 1), I.Matrix("one", 1, 64, 0, 2)]
    q = pq.PQ_LSQ4
    peers = LocalPeers(world)
    ranks = [ShardedQuantStep(mats, q, k, world, peers, device=DEV) for k in range(world)]
    one = []
    for i, m in enumerate(mats):
        w = I.normal_weights(m.rows, m.cols, seed=i, stream=0, device=DEV)
        a = I.alpha_init(w, q)
        g = I.grad_bf16(m.rows, m.cols, seed=9, stream=i, device=DEV)
        for r in ranks:
            r.load_full(i, w, a)
            r.g(i).copy_(g)  # equal replicas: their mean is g
        z = lambda *s: torch.zeros(*s, device=DEV)
        one.append(dict(rows=m.rows, cols=m.cols, w=w.clone(), alpha=a.clone(), g=g, m_w=z(m.rows, m.cols),
                        v_w=z(m.rows, m.cols), m_alpha=z(m.rows), v_alpha=z(m.rows),
                        grad_scale=pq.pq_default_grad_scale(q, m.cols)))
    hw, ha = pq.adamw(1, 1e-4), pq.adamw(1, 1e-5)
    norm, coef = outs()
    pq.pq_grad_norm(0.01, norm, coef, scratch(pq, 0, len(one)), q=q, mats=pq.matrix_array(one))
    pq.pq_fakequant_bwd_adamw(q, pq.adamw_matrix_array(one), hw, ha, coef=coef)
    sums = torch.zeros(world, dtype=torch.float64, device=DEV)
    for r in ranks:  # every rank's sum before any rank's update
        sources, mult, shards = r._reduce_args(None)
        pq.pq_reduce_grad_norm(q, sources, mult, shards, 0.01, None, None, scratch(pq, 0, len(mats)),
                               sumsq_out=sums[r.rank:r.rank + 1])
    for r in ranks:
        got, c = r.clip_coef(0.01, gather=lambda s: sums)
        # both add the same squares, in another order
        assert float(got) == pytest.approx(float(norm), rel=RTOL)
        assert float(c) == pytest.approx(float(coef), rel=RTOL)
        r.reduce_step(hw, ha, coef=coef)
    for i, m in enumerate(mats):
        for r in ranks:
            b, e = r.my_rows(i)
            assert torch.equal(r.w_shard(i), one[i]["w"][b:e])
            assert torch.equal(r.alpha_rows(i, b, e), one[i]["alpha"][b:e])


def test_quant_step_norm_and_clip(pq):
    from bit_quantization_aware_b200.step import QuantStep
    mats = [I.Matrix("a", 256, 512, 0, 0), I.Matrix("b", 33, 72, 0, 1)]
    st = QuantStep(mats, pq.PQ_SEQ2, device=DEV)
    st.generate(seed=3)
    st.run()
    grads = [t.clone() for b in st.bufs for t in (b.dw, b.dalpha)]
    want = norm64(grads)
    norm, coef = st.grad_norm(0.25 * want)
    assert float(norm) == pytest.approx(want, rel=RTOL)
    assert float(coef) == pytest.approx(coef_of(want, 0.25 * want), rel=RTOL)
    c = coef.clone()
    norm = st.clip_grads(0.25 * want)
    assert float(norm) == pytest.approx(want, rel=RTOL)
    for t, k in zip([t for b in st.bufs for t in (b.dw, b.dalpha)], grads):
        # the two norms may round differently: factors within an fp32 step
        assert torch.allclose(t, k * c, rtol=2.0 ** -22, atol=0)


@pytest.mark.parametrize("as_int", [False, True])
def test_clipping_workspace_belongs_to_the_stream(pq, monkeypatch, as_int):
    """clip_grad_norm returns while its kernels run: the workspace that it
    gives back must not go to the current stream's next allocation."""
    ts = [torch.randn(n, generator=torch.Generator().manual_seed(n)).to("cuda") for n in (5, 4096, 100001)]
    want = float(torch.cat([t.double() for t in ts]).norm())
    torch.cuda.synchronize()
    seen = []
    call = pq.pq_grad_clip
    monkeypatch.setattr(pq, "pq_grad_clip", lambda *a: (seen.append((a[2], a[4].data_ptr(), a[4].numel())), call(*a)))
    side = torch.cuda.Stream()
    norm = pq.clip_grad_norm(ts, 1.0, side.cuda_stream if as_int else side)
    _, at, size = seen[0]
    taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != at for t in taken)
    side.synchronize()
    # the norm: fp64 sums rounded once to fp32
    assert abs(float(norm) - want) <= want * (torch.finfo(torch.float32).eps / 2 + 1e-12)
