"""The training-step operators around the weight quantizer, measured.

Four operators: block quantization to e4m3 ("quant"), the matrix product of
two block-quantized operands ("gemm", alone and as the three products of one
linear layer's step, "linear"), the global gradient norm with clipping
("clip") and the quantizer's own gradient norm followed by the clipped
backward + AdamW ("step"). Sizes are the linear layers of the 1B-class and
Llama-3-8B-shaped sets, and ragged ones between them.

``run`` computes each in its plain form (elementary torch operations) or,
where ``own`` is true, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
FMAX = 448.0            # largest finite e4m3
TINY = 2.0 ** -96       # smallest block maximum a scale is made from
CLIP = 0.9900000095367432  # the quantizers' 0.99 in fp32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
QUANTIZERS = ("binary", "ternary", "seq2", "seq2_b", "lsq2", "lsq3", "lsq4")
LSQ = {"lsq2": (-2, 1), "lsq3": (-4, 3), "lsq4": (-8, 7)}
QP = {"binary": 1.0, "ternary": 1.0, "lsq2": 1.0, "seq2": 1.5, "seq2_b": 1.5, "lsq3": 3.0, "lsq4": 7.0}
# AdamW of the weights and of the scales, whose rate is lower so that they stay positive over many passes
HP = {"lr": 2e-5, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.0, "step": 100}
HP_ALPHA = dict(HP, lr=5e-7)


def listed():
    return [
        # activations of a decode batch, quantized by rows in front of a product
        {"name": "quant_rows_16x4096", "kind": "quant", "rows": 16, "cols": 4096, "dtype": "bf16", "block": "row", "transposed": False},
        # a training batch's activations: by rows for the forward product, by columns for the weight gradient
        {"name": "quant_both_8192x4096", "kind": "quant", "rows": 8192, "cols": 4096, "dtype": "bf16", "block": "row", "transposed": True},
        # the gate projection's fake-quantized weights in 128 x 128 blocks, with the transpose the input gradient reads
        {"name": "quant_tiles_14336x4096", "kind": "quant", "rows": 14336, "cols": 4096, "dtype": "bf16", "block": "tile", "transposed": True},
        # one token through the o projection
        {"name": "gemm_1x4096x4096", "kind": "gemm", "m": 1, "n": 4096, "k": 4096, "b": "tile", "out": "bf16"},
        # an odd batch of tokens through the gate projection
        {"name": "gemm_77x14336x4096", "kind": "gemm", "m": 77, "n": 14336, "k": 4096, "b": "tile", "out": "bf16"},
        # a training batch through the gate projection
        {"name": "gemm_8192x14336x4096", "kind": "gemm", "m": 8192, "n": 14336, "k": 4096, "b": "tile", "out": "bf16"},
        # the o projection's weight gradient over a ragged number of tokens, in fp32
        {"name": "gemm_4096x4096x8190", "kind": "gemm", "m": 4096, "n": 4096, "k": 8190, "b": "row", "out": "fp32"},
        # a whole step of the 1B-class up projection: quantize weights, activations and the output's gradient, three products
        {"name": "linear_4096x5632x2048", "kind": "linear", "m": 4096, "n": 5632, "k": 2048},
        # the norm weights and scales of a 24-layer model: many short vectors
        {"name": "clip_98_short", "kind": "clip", "lengths": "98x2048", "dtype": "fp32", "out": "fp32"},
        # the linear layers' bf16 gradients of eight Llama-3-8B-shaped layers, into fp32
        {"name": "clip_56_long", "kind": "clip", "lengths": "16x16777216,16x4194304,24x58720256", "dtype": "bf16", "out": "fp32"},
        # one small matrix: the clipped quantizer backward and AdamW
        {"name": "step_256x1024", "kind": "step", "q": "seq2", "shapes": "1x256x1024"},
        # two Llama-3-8B-shaped layers: the same
        {"name": "step_2_layers", "kind": "step", "q": "seq2", "shapes": "4x4096x4096,4x1024x4096,4x14336x4096,2x4096x14336"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("quant", "quant", "gemm", "gemm", "gemm", "linear", "clip", "step"))
    if kind == "quant":
        return {"kind": kind, "rows": _log(rng, 1, 14336), "cols": _log(rng, 16, 14336), "dtype": rng.choice(("bf16", "fp16", "fp32")),
                "block": rng.choice(("row", "tile")), "transposed": rng.random() < 0.5}
    if kind == "gemm":
        return {"kind": kind, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 14336), "k": _log(rng, 64, 8192) // 2,
                "b": rng.choice(("tile", "tile", "row")), "out": rng.choice(("bf16", "bf16", "fp32", "fp16"))}
    if kind == "linear":
        return {"kind": kind, "m": _log(rng, 16, 8192), "n": _log(rng, 128, 5632), "k": _log(rng, 128, 5632)}
    if kind == "clip":
        dtype = rng.choice(("bf16", "fp16", "fp32"))
        lengths = ",".join("%dx%d" % (_log(rng, 1, 60), _log(rng, 1, 1 << 23)) for _ in range(rng.randint(1, 4)))
        return {"kind": kind, "lengths": lengths, "dtype": dtype, "out": rng.choice((dtype, "fp32"))}
    shapes = ",".join("%dx%dx%d" % (_log(rng, 1, 6), _log(rng, 1, 4096), _log(rng, 1, 8192)) for _ in range(rng.randint(1, 3)))
    return {"kind": kind, "q": rng.choice(QUANTIZERS), "shapes": shapes}


def _blocks(v):
    return (v + 127) // 128


def _lengths(text):
    return [int(x) for part in text.split(",") for n, x in (part.split("x"),) for _ in range(int(n))]


def _shapes(text):
    return [(int(r), int(c)) for part in text.split(",") for n, r, c in (part.split("x"),) for _ in range(int(n))]


def _offsets(sizes):
    """Places of tensors in one flat buffer, each on a multiple of 64 elements, and its length."""
    at, total = [], 0
    for s in sizes:
        at.append(total)
        total += (s + 63) // 64 * 64
    return at, total


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _activations(rows, cols, dtype, g):
    """Normal values with a few channels twenty times the others, as hidden states have them."""
    x = torch.randn(rows, cols, device=DEV, generator=g)
    x *= torch.where(torch.rand(cols, device=DEV, generator=g) < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _weights(rows, cols, g):
    """Fake-quantized weights: the 2-bit SEQ levels times a scale for each row."""
    alpha = 0.05 * (1 + 0.2 * torch.rand(rows, 1, device=DEV, generator=g))
    level = torch.randint(0, 4, (rows, cols), device=DEV, generator=g).float() * 0.5 - 0.75
    return (level * alpha).to(torch.bfloat16)


def _padded(codes):
    """Codes with a row pitch of a multiple of 16 bytes, as the quantization writes them."""
    rows, cols = codes.shape
    q = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device=codes.device).view(torch.float8_e4m3fn)[:, :cols]
    return q.copy_(codes)


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    if kind == "quant":
        make = _weights if case["block"] == "tile" else lambda r, c, gen: _activations(r, c, torch.float32, gen)
        return dict(case, x=make(case["rows"], case["cols"], g).to(DTYPES[case["dtype"]]))
    if kind == "gemm":
        a, sa = _quant_rows(_activations(case["m"], case["k"], torch.float32, g))
        if case["b"] == "tile":
            b, sb = _quant_tiles(_weights(case["n"], case["k"], g).float())
        else:
            b, sb = _quant_rows(1e-3 * _activations(case["n"], case["k"], torch.float32, g))
        return dict(case, a=_padded(a), sa=sa, bq=_padded(b), sb=sb)
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s = dict(case, x=_activations(m, k, torch.bfloat16, g), w=_weights(n, k, g), dy=(1e-3 * torch.randn(m, n, device=DEV, generator=g)).to(torch.bfloat16))
        if own:
            from bit_quantization_aware_b200.linear import Fp8Linear
            s["layer"] = Fp8Linear(n, k, m, device=DEV)
        return s
    if kind == "clip":
        sizes = _lengths(case["lengths"])
        at, total = _offsets(sizes)
        flat = (1e-3 * torch.randn(total, device=DEV, generator=g)).to(DTYPES[case["dtype"]])
        out = torch.zeros(total, device=DEV, dtype=DTYPES[case["out"]])
        for o, n, nxt in zip(at, sizes, at[1:] + [total]):
            flat[o + n:nxt] = 0  # between the tensors
        s = dict(case, flat=flat, out_flat=out, max_norm=0.25)
        s["grads"] = [flat[o:o + n] for o, n in zip(at, sizes)]
        s["outs"] = [out[o:o + n] for o, n in zip(at, sizes)]
        if own:
            from bit_quantization_aware_b200 import pq
            s["tensors"] = pq.tensor_array(s["grads"], s["outs"])
            s["scratch"] = torch.empty(pq.pq_grad_norm_workspace_bytes(len(sizes), 0), dtype=torch.uint8, device=DEV)
            s["norm"], s["coef"] = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        return s
    shapes = _shapes(case["shapes"])
    at, total = _offsets([r * c for r, c in shapes])
    rat, rtotal = _offsets([r for r, _ in shapes])
    w = 0.02 * torch.randn(total, device=DEV, generator=g)
    grad = (1e-3 * torch.randn(total, device=DEV, generator=g)).to(torch.bfloat16)
    m_w = 1e-4 * torch.randn(total, device=DEV, generator=g)
    v_w = 1e-7 * (0.1 + torch.rand(total, device=DEV, generator=g))
    alpha = torch.ones(rtotal, device=DEV)
    m_a = 1e-4 * torch.randn(rtotal, device=DEV, generator=g)
    v_a = 1e-7 * (0.1 + torch.rand(rtotal, device=DEV, generator=g))
    s = dict(case, w=w, g=grad, m_w=m_w, v_w=v_w, alpha=alpha, m_a=m_a, v_a=v_a, max_norm=0.1, mats=[])
    for (r, c), o, ro in zip(shapes, at, rat):
        v = {"rows": r, "cols": c, "grad_scale": 1.0 / math.sqrt(c * QP[case["q"]])}
        for key, flat in (("w", w), ("g", grad), ("m_w", m_w), ("v_w", v_w)):
            v[key] = flat[o:o + r * c].view(r, c)
        for key, flat in (("alpha", alpha), ("m_alpha", m_a), ("v_alpha", v_a)):
            v[key] = flat[ro:ro + r]
        mag = v["w"].abs()
        v["alpha"].copy_(2 * mag.mean(1) / math.sqrt(QP[case["q"]]) if case["q"] in LSQ or case["q"] == "binary" else mag.amax(1).clamp_min(1e-6))
        s["mats"].append(v)
    if own:
        from bit_quantization_aware_b200 import pq
        s["norm_mats"], s["adamw_mats"] = pq.matrix_array(s["mats"]), pq.adamw_matrix_array(s["mats"])
        s["hp"], s["hp_alpha"] = pq.adamw(**HP), pq.adamw(**HP_ALPHA)
        s["scratch"] = torch.empty(pq.pq_grad_norm_workspace_bytes(0, len(shapes)), dtype=torch.uint8, device=DEV)
        s["norm"], s["coef"] = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    return s


# ------------------------------------------------------------ plain forms
def _scales(amax):
    amax = amax.clamp_min(TINY)
    top = torch.full_like(amax, FMAX)  # a number over a tensor would be its reciprocal times the number
    return amax / top, top / amax


def _round_e4m3(v):
    return v.clamp(-FMAX, FMAX).to(torch.float8_e4m3fn)


def _quant_rows(x):
    """One scale for each 128 consecutive values of a row: e4m3 codes [rows, cols] and scales [blocks, rows]."""
    rows, cols = x.shape
    kb = _blocks(cols)
    p = torch.zeros(rows, kb * 128, device=x.device)
    p[:, :cols] = x
    p = p.view(rows, kb, 128)
    s, r = _scales(p.abs().amax(2))
    q = _round_e4m3(p * r[:, :, None]).view(rows, kb * 128)[:, :cols]
    return q, s.t().contiguous()


def _quant_tiles(x):
    """One scale for each 128 x 128 block: codes [rows, cols] and scales [row blocks, column blocks]."""
    rows, cols = x.shape
    rb, cb = _blocks(rows), _blocks(cols)
    p = torch.zeros(rb * 128, cb * 128, device=x.device)
    p[:rows, :cols] = x
    p = p.view(rb, 128, cb, 128)
    s, r = _scales(p.abs().amax(3).amax(1))
    q = _round_e4m3(p * r[:, None, :, None]).view(rb * 128, cb * 128)[:rows, :cols]
    return q, s


def _values(q, s, block):
    """What codes and scales stand for, in the scales' type."""
    rows, cols = q.shape
    if block == "row":
        f = s.t().repeat_interleave(128, 1)[:, :cols]
    else:
        f = s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q.to(s.dtype) * f


def _quant(x, block, transposed):
    f = _quant_rows if block == "row" else _quant_tiles
    out = list(f(x.float()))
    if transposed:
        out += f(x.float().t())
    return out


def _linear(s):
    x, w, dy = s["x"], s["w"], s["dy"]
    xr, xc = _values(*_quant_rows(x.float()), "row"), _values(*_quant_rows(x.float().t()), "row")
    yr, yc = _values(*_quant_rows(dy.float()), "row"), _values(*_quant_rows(dy.float().t()), "row")
    wt = _values(*_quant_tiles(w.float()), "tile")
    return {"y": (xr @ wt.t()).to(torch.bfloat16), "dx": (yr @ wt).to(torch.bfloat16), "dw": (yc @ xc.t()).to(torch.bfloat16)}


def _coef(sumsq, max_norm):
    norm = sumsq.sqrt()
    return norm, (max_norm / (norm + 1e-6)).clamp_max(1.0)


def _clip(s):
    norm, coef = _coef(sum(t.double().square().sum() for t in s["grads"]), s["max_norm"])
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * coef.float())
    return {"norm": norm.float().view(1), "grads": s["out_flat"]}


def _level(q, x):
    """The quantizer's level in units of alpha, and whether x is inside its clipping range."""
    if q == "binary":
        return torch.where(x >= 0, 1.0, -1.0).to(x.dtype), x.abs() <= 1.0
    if q in LSQ:
        lo, hi = LSQ[q]
        return x.clamp(lo, hi).round(), (x >= lo) & (x <= hi)
    c = x.clamp(-CLIP, CLIP)
    if q == "ternary":
        level = (c * 1.5).round() / 1.5
    elif q == "seq2":
        level = ((c * 2 - 0.5).round() + 0.5) / 2
    else:
        level = ((c * 1.5 - 0.5).round() + 0.5) / 1.5
    return level, x.abs() <= CLIP


def _adamw(p, m, v, g, hp):
    m.mul_(hp["beta1"]).add_(g * (1 - hp["beta1"]))
    v.mul_(hp["beta2"]).add_(g * g * (1 - hp["beta2"]))
    den = v.sqrt() * (1 / math.sqrt(1 - hp["beta2"] ** hp["step"])) + hp["eps"]
    p.sub_(m / den * (hp["lr"] / (1 - hp["beta1"] ** hp["step"])))


def _quantizer_grads(q, v):
    """dW and d(alpha) of one matrix."""
    x = v["w"] / v["alpha"][:, None]
    level, inside = _level(q, x)
    g = v["g"].float()
    da = (g.double() * (level.double() - torch.where(inside, x, 0.0).double())).sum(1) * v["grad_scale"]
    return torch.where(inside, g, 0.0), da.float()


def _step(s):
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for v in s["mats"]:
        dw, da = _quantizer_grads(s["q"], v)
        total += dw.double().square().sum() + da.double().square().sum()
    norm, coef = _coef(total, s["max_norm"])
    for v in s["mats"]:
        dw, da = _quantizer_grads(s["q"], v)
        _adamw(v["w"], v["m_w"], v["v_w"], dw * coef.float(), HP)
        _adamw(v["alpha"], v["m_alpha"], v["v_alpha"], da * coef.float(), HP_ALPHA)
    return _step_outputs(s, norm.float().view(1))


def _step_outputs(s, norm):
    return {"norm": norm, "w": s["w"], "m_w": s["m_w"], "v_w": s["v_w"], "alpha": s["alpha"], "m_a": s["m_a"], "v_a": s["v_a"]}


def _plain(s):
    kind = s["kind"]
    if kind == "quant":
        return _quant(s["x"], s["block"], s["transposed"])
    if kind == "gemm":
        return (_values(s["a"], s["sa"], "row") @ _values(s["bq"], s["sb"], s["b"]).t()).to(DTYPES[s["out"]])
    return {"linear": _linear, "clip": _clip, "step": _step}[kind](s)


# -------------------------------------------------------- the library's calls
def _call(s):
    from bit_quantization_aware_b200 import pq
    kind = s["kind"]
    if kind == "quant":
        block = pq.PQ_BLOCK_ROW if s["block"] == "row" else pq.PQ_BLOCK_TILE
        out = pq.fp8_quant(s["x"], block, transposed=s["transposed"])
        return list(out) if s["transposed"] else list(out[:2])
    if kind == "gemm":
        block = pq.PQ_BLOCK_ROW if s["b"] == "row" else pq.PQ_BLOCK_TILE
        return pq.fp8_gemm(s["a"], s["sa"], s["bq"], s["sb"], block, out_dtype=DTYPES[s["out"]])
    if kind == "linear":
        y = s["layer"].forward(s["x"], s["w"])
        dx, dw = s["layer"].backward(s["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    if kind == "clip":
        pq.pq_grad_clip(s["tensors"], s["max_norm"], s["norm"], s["coef"], s["scratch"])
        return {"norm": s["norm"], "grads": s["out_flat"]}
    q = pq.QUANTIZERS[s["q"]]
    pq.pq_grad_norm(s["max_norm"], s["norm"], s["coef"], s["scratch"], q=q, mats=s["norm_mats"])
    pq.pq_fakequant_bwd_adamw(q, s["adamw_mats"], s["hp"], s["hp_alpha"], coef=s["coef"])
    return _step_outputs(s, s["norm"])


def run(state):
    return _call(state) if own else _plain(state)


# --------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if kind == "quant":
        r, c = case["rows"], case["cols"]
        ways = [(r, c), (c, r)] if case["transposed"] else [(r, c)]
        scales = sum(_blocks(b) * a if case["block"] == "row" else _blocks(a) * _blocks(b) for a, b in ways)
        return {"bytes": r * c * (size[case["dtype"]] + len(ways)) + 4 * scales, "flops": 4 * r * c}
    if kind == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        sb = _blocks(k) * (n if case["b"] == "row" else _blocks(n))
        return {"bytes": (m + n) * k + 4 * _blocks(k) * m + 4 * sb + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        # x, w, dy read and y, dx, dw written in bf16; the codes between them need not reach memory
        return {"bytes": 4 * (m * k + n * k + m * n), "flops": 6 * m * n * k}
    if kind == "clip":
        total = sum(_lengths(case["lengths"]))
        return {"bytes": total * (size[case["dtype"]] + size[case["out"]]) + 4, "flops": 3 * total}
    weights = sum(r * c for r, c in _shapes(case["shapes"]))
    rows = sum(r for r, _ in _shapes(case["shapes"]))
    return {"bytes": 26 * weights + 24 * rows, "flops": 40 * weights}


# ------------------------------------------------ the definitions in 64 bits
def _nearest_e4m3(v):
    """The e4m3 value nearest to each v, ties to even; beyond 448, 448."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-FMAX, FMAX)


def _exact_quant(x, block):
    """Codes as the values they stand for and scales, each block on its own."""
    rows, cols = x.shape
    tall = 1 if block == "row" else 128
    rb, cb = (rows + tall - 1) // tall, _blocks(cols)
    amax = torch.nn.functional.pad(x.abs(), (0, cb * 128 - cols, 0, rb * tall - rows)).reshape(rb, tall, cb, 128).amax((1, 3)).clamp_min(TINY)
    of_row = torch.arange(rows, device=x.device) // tall
    of_col = torch.arange(cols, device=x.device) // 128
    q = _nearest_e4m3(x * FMAX / amax[of_row][:, of_col])
    s = amax / FMAX
    return q, s.t() if block == "row" else s


def _exact_values(q, s, block):
    n = torch.arange(q.shape[0], device=q.device)
    k = torch.arange(q.shape[1], device=q.device) // 128
    return q.double() * (s.double().t()[:, k] if block == "row" else s.double()[n // 128][:, k])


def _exact_step(s):
    grads, total = [], 0.0
    for v in s["mats"]:
        x = v["w"].double() / v["alpha"].double()[:, None]
        g = v["g"].double()
        level, inside = _level(s["q"], x)
        da = (g * (level - x * inside)).sum(1) * v["grad_scale"]
        grads.append((g * inside, da))
        total = total + (g * inside).pow(2).sum() + da.pow(2).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    out = {key: s[key].double() for key in ("w", "m_w", "v_w", "alpha", "m_a", "v_a")}
    at, rat = 0, 0
    c1, c2 = 1 - HP["beta1"] ** HP["step"], 1 - HP["beta2"] ** HP["step"]
    for v, (dw, da) in zip(s["mats"], grads):
        for p, m, u, o, g, lr in (("w", "m_w", "v_w", at, dw.flatten(), HP["lr"]), ("alpha", "m_a", "v_a", rat, da, HP_ALPHA["lr"])):
            here = slice(o, o + g.numel())
            out[m][here] = HP["beta1"] * out[m][here] + (1 - HP["beta1"]) * coef * g
            out[u][here] = HP["beta2"] * out[u][here] + (1 - HP["beta2"]) * (coef * g) ** 2
            out[p][here] -= lr * (out[m][here] / c1) / ((out[u][here] / c2).sqrt() + HP["eps"])
        at += (v["rows"] * v["cols"] + 63) // 64 * 64
        rat += (v["rows"] + 63) // 64 * 64
    return {"norm": norm.view(1), **out}


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind == "quant":
        x = s["x"].double()
        return [t for v in ([x, x.t()] if case["transposed"] else [x]) for t in _exact_quant(v, case["block"])]
    if kind == "gemm":
        return _exact_values(s["a"], s["sa"], "row") @ _exact_values(s["bq"], s["sb"], case["b"]).t()
    if kind == "linear":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        xr, xc, yr, yc = (_exact_values(*_exact_quant(t, "row"), "row") for t in (x, x.t(), dy, dy.t()))
        wt = _exact_values(*_exact_quant(w, "tile"), "tile")
        return {"y": xr @ wt.t(), "dx": yr @ wt, "dw": yc @ xc.t()}
    if kind == "clip":
        norm = torch.stack([torch.linalg.vector_norm(t, dtype=torch.float64) for t in s["grads"]]).square().sum().sqrt()
        coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        out = torch.zeros(s["flat"].numel(), dtype=torch.float64, device=DEV)
        at, _ = _offsets([t.numel() for t in s["grads"]])
        for o, t in zip(at, s["grads"]):
            out[o:o + t.numel()] = t.double() * coef
        return {"norm": norm.view(1), "grads": out}
    return _exact_step(s)
