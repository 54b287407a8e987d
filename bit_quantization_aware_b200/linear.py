"""The three products of a linear layer's training step in block-scaled e4m3.

Around the weight quantizer, a step of one layer y = x Wq^T multiplies three
times: y from the activations and the fake-quantized weights, dx from the
output's gradient and the weights, and the weights' upstream gradient
dWq = dy^T x, which the quantizer's backward takes (``pq_fakequant_bwd``,
``pq_fakequant_bwd_adamw``). ``Fp8Linear`` quantizes each operand once
(``pq.pq_fp8_quant``: x and dy by rows and, from the same read, by columns;
Wq in 128 x 128 tiles with its transpose) and runs the products on the tensor
cores (``pq.pq_fp8_gemm``). It holds the codes between forward and backward
and allocates nothing but the outputs that the caller leaves out.

Every operand is rounded to e4m3 (three mantissa bits) on the way, Wq among
them: the products are those of the codes, x' W'^T and so on, not of Wq to the
bit. A row's levels are multiples of its own alpha while a tile has one scale
for 128 rows, so the levels fall between codes: of normal weights with the
quantizers' initial alphas, W' is 2.0 to 2.7% from Wq (root mean square;
single weights up to 5.9%, never more than 2^-4), and the packed codes do not
hold W'. Where the weights that are served have to be multiplied as they are,
take a bf16 product of Wq or ``pq_wq_gemm`` of the packed codes.
"""
from __future__ import annotations

import torch

from . import pq


class _Operand:
    """Codes and scales of one operand and of its transpose, for up to
    ``rows`` x ``cols``; ``quant`` fills and returns views of the size at hand."""

    def __init__(self, block, rows, cols, device):
        self.block, self.rows, self.cols = block, rows, cols
        self.q = pq.fp8_empty(rows, cols, device)
        self.qt = pq.fp8_empty(cols, rows, device)
        count = lambda r, c: torch.Size(pq.fp8_scale_shape(block, r, c)).numel()
        self.s = torch.empty(count(rows, cols), dtype=torch.float32, device=device)
        self.st = torch.empty(count(cols, rows), dtype=torch.float32, device=device)
        self._size, self._views = None, None

    def _views_of(self, r, c):
        shape, shape_t = pq.fp8_scale_shape(self.block, r, c), pq.fp8_scale_shape(self.block, c, r)
        return ((self.q[:r], self.s[:shape[0] * shape[1]].view(shape)),
                (self.qt[:, :r], self.st[:shape_t[0] * shape_t[1]].view(shape_t)))

    def quant(self, x, stream):
        size = tuple(x.shape)
        # the last size's views stand: making a forward's two sets anew takes
        # 17 us of host time
        if size != self._size:
            self._size, self._views = size, self._views_of(*size)
        (q, s), (qt, st) = self._views
        pq.pq_fp8_quant(self.block, x, q, s, qt, st, stream)
        return self._views


class Fp8Linear:
    """One linear layer of ``out_features`` x ``in_features`` weights over up
    to ``max_tokens`` tokens a step, its operands rounded to e4m3 (how far
    that is from x Wq^T: see the module)."""

    def __init__(self, out_features, in_features, max_tokens, device="cuda"):
        if min(out_features, in_features, max_tokens) < 1:
            raise ValueError("Fp8Linear: sizes must be positive")
        self.n, self.k, self.max_tokens = int(out_features), int(in_features), int(max_tokens)
        dev = torch.device(device)
        self._w = _Operand(pq.PQ_BLOCK_TILE, self.n, self.k, dev)
        self._x = _Operand(pq.PQ_BLOCK_ROW, self.max_tokens, self.k, dev)
        self._dy = _Operand(pq.PQ_BLOCK_ROW, self.max_tokens, self.n, dev)
        self._saved = None  # (tokens, W^T codes, x^T codes) of the last forward

    def _check(self, t, rows, cols, name):
        if t.dim() != 2 or tuple(t.shape) != (rows, cols):
            raise ValueError(f"Fp8Linear: {name} must be [{rows}, {cols}], got {list(t.shape)}")

    @staticmethod
    def _out(rows, cols, like, stream):
        return pq._new(like, (rows, cols), torch.bfloat16, stream)

    def forward(self, x, wq, y_out=None, stream=None):
        """y = x Wq^T of the operands' e4m3 codes (bf16 [tokens,
        out_features], or ``y_out``'s type) from x [tokens, in_features] and
        wq [out_features, in_features]."""
        m = x.shape[0]
        if not 1 <= m <= self.max_tokens:
            raise ValueError(f"Fp8Linear: 1 to {self.max_tokens} tokens, got {m}")
        self._check(x, m, self.k, "x")
        self._check(wq, self.n, self.k, "wq")
        self._saved = None  # its codes are overwritten from here on
        w, wt = self._w.quant(wq, stream)
        xr, xt = self._x.quant(x, stream)
        y = y_out if y_out is not None else self._out(m, self.n, x, stream)
        pq.pq_fp8_gemm(*xr, *w, pq.PQ_BLOCK_TILE, y, stream)
        self._saved = (m, wt, xt)
        return y

    def backward(self, dy, dx_out=None, dw_out=None, stream=None):
        """(dx [tokens, in_features], dWq [out_features, in_features]) of the
        last forward, bf16 unless given, from dy [tokens, out_features]."""
        if self._saved is None:
            raise ValueError("Fp8Linear: backward needs a forward first")
        m, wt, xt = self._saved
        self._check(dy, m, self.n, "dy")
        dyr, dyt = self._dy.quant(dy, stream)
        dx = dx_out if dx_out is not None else self._out(m, self.k, dy, stream)
        dw = dw_out if dw_out is not None else self._out(self.n, self.k, dy, stream)
        pq.pq_fp8_gemm(*dyr, *wt, pq.PQ_BLOCK_TILE, dx, stream)
        pq.pq_fp8_gemm(*dyt, *xt, pq.PQ_BLOCK_ROW, dw, stream)
        return dx, dw
