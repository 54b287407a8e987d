"""Block quantization to e4m3 and the block-scaled product in 64 bits, from
their definitions, on the CPU: what the CUDA kernels are compared with."""
from __future__ import annotations

import torch

ROW, TILE = 1, 2


def e4m3(v: torch.Tensor) -> torch.Tensor:
    """The e4m3 value nearest to each fp64 v (ties to even), saturating at
    448; NaN stays NaN."""
    e = torch.frexp(v.abs().clamp(2.0 ** -20, 1e30))[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def amax(x: torch.Tensor, block: int) -> torch.Tensor:
    """Largest magnitude of each block, not below 2^-96: [blocks, rows] (ROW)
    or [row blocks, column blocks] (TILE)."""
    rows, cols = x.shape
    tall = 1 if block == ROW else 128
    out = torch.stack([torch.stack([x[r:r + tall, c:c + 128].abs().max() for c in range(0, cols, 128)])
                       for r in range(0, rows, tall)]).clamp_min(2.0 ** -96)
    return out.t().contiguous() if block == ROW else out


def expand(s: torch.Tensor, block: int, rows: int, cols: int) -> torch.Tensor:
    """A scale for every element."""
    k = torch.arange(cols) // 128
    return s.t()[:, k] if block == ROW else s[torch.arange(rows) // 128][:, k]


def quant(x: torch.Tensor, block: int):
    """Codes' values and scales with the fp32 steps of the definition: the
    kernel's results are these bit for bit."""
    f = x.float().cpu()
    m = amax(f, block)
    top = torch.full_like(m, 448.0)  # a number over a tensor would be its reciprocal times the number
    s, r = m / top, top / m
    v = f * expand(r, block, *f.shape)  # fp32, rounded once
    return e4m3(v.double()), s


def values(q: torch.Tensor, s: torch.Tensor, block: int) -> torch.Tensor:
    q = q.cpu()
    if q.dtype == torch.uint8:
        q = q.view(torch.float8_e4m3fn)
    return q.float().double() * expand(s.cpu().double(), block, *q.shape)


def product(a, sa, b, sb, b_block):
    """Y in fp64 and the sum of its terms' magnitudes."""
    va, vb = values(a, sa, ROW), values(b, sb, b_block)
    return va @ vb.t(), va.abs() @ vb.abs().t()


def product_tolerance(y, mags, k, dtype):
    """How far an element of the product may be off. Within a block the
    products are exact in fp32 and each of the 128 additions is off by at
    most one step (2^-23) of the block's partial sum, whether it rounds or
    cuts; the scale's product, the scaling and the sum over the blocks round
    to nearest (2^-24 each); the output rounds by half a step of its type."""
    blocks = (k + 127) // 128
    return mags * (128 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24) + y.abs() * torch.finfo(dtype).eps / 2 + \
        torch.finfo(dtype).tiny
