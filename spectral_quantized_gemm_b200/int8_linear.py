"""Linear layer on 8-bit integer operands, for training and serving.

``Int8Linear`` computes ``Y = X W`` (X: tokens x in_features, W: in_features x
out_features, as ``MetisLinear``) with 8-bit integer products inside libmetis, one scale
for each line of both operands that is not contracted:

  forward   Y  = Q(X) Q(W)          scales for each token and each output channel
  backward  dX = Q(dY) Q(W)^T       scales for each token and each input channel
            dW = Q(X)^T Q(dY)       scales for each input and each output channel

Every operand is quantized (round to nearest) along the dimension that its product
contracts, so the forward and backward products read different codes of the same matrix.
The sums are exact 32-bit integers.  The layer keeps an fp32 master weight; Y is bf16, dX has
the type of X and dW is fp32 (cast to the weight's type).  Between forward and backward it
keeps the codes of X and W, not X itself.

Serving: ``freeze()`` lays the 8-bit weight out once; calls without gradients then read it
instead of quantizing the weight each time, until ``unfreeze()``.

Any number of tokens and features is allowed (in_features, and out_features and tokens of
a backward pass, up to 131071, the bound of the exact sum).  There is no CPU path.
"""

import math

import torch

from . import Int8
from .linear import _shared_context

MAX_INNER = 131071


def _output(rows, cols, dtype, device):
    """rows x cols with rows that start on 16 bytes."""
    size = 8 if dtype == torch.bfloat16 else 4
    return torch.empty(rows, -(-cols // size) * size, dtype=dtype, device=device)[:, :cols]


def _operand(M):
    """M as the quantizer reads it: fp32 or bf16, unit stride along a row."""
    if M.dtype not in (torch.float32, torch.bfloat16):
        M = M.float()
    return M if M.stride(-1) == 1 or M.shape[-1] == 1 else M.contiguous()


class _Int8LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        need_dx, need_dw = ctx.needs_input_grad
        rows, (m, n) = x.shape[0], weight.shape
        ctx.x_dtype, ctx.w_dtype, ctx.sizes = x.dtype, weight.dtype, (rows, m, n)
        if rows == 0:
            return torch.empty(0, n, dtype=torch.bfloat16, device=x.device)
        x, w = _operand(x), _operand(weight)
        lib, lock = _shared_context(x.device)
        with lock:
            xr, xc = lib.new_int8(rows, m), lib.new_int8(m, rows) if need_dw else None
            wr, wc = lib.new_int8(m, n) if need_dx else None, lib.new_int8(n, m)
            lib.quantize_int8(x, rowwise=xr, colwise=xc)
            lib.quantize_int8(w, rowwise=wr, colwise=wc)
            y = _output(rows, n, torch.bfloat16, x.device)
            lib.gemm_int8(xr, wc, y)
        ctx.save_for_backward(*(t for q in (xc, wr) if q is not None for t in (q.codes, q.scales)))
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_dx, need_dw = ctx.needs_input_grad
        rows, m, n = ctx.sizes
        if rows == 0:
            return (torch.empty(0, m, dtype=ctx.x_dtype, device=dy.device) if need_dx else None,
                    torch.zeros(m, n, dtype=ctx.w_dtype, device=dy.device) if need_dw else None)
        saved = list(ctx.saved_tensors)
        dy = _operand(dy)
        lib, lock = _shared_context(dy.device)
        dx = dw = None
        with lock:
            dr = lib.new_int8(rows, n) if need_dx else None
            dc = lib.new_int8(n, rows) if need_dw else None
            lib.quantize_int8(dy, rowwise=dr, colwise=dc)
            if need_dw:
                xc = Int8(m, rows, codes=saved[0], scales=saved[1])
                dw = _output(m, n, torch.float32, dy.device)
                lib.gemm_int8(xc, dc, dw)
            if need_dx:
                wr = Int8(m, n, codes=saved[-2], scales=saved[-1])
                dx = _output(rows, m, torch.float32 if ctx.x_dtype != torch.bfloat16 else torch.bfloat16, dy.device)
                lib.gemm_int8(dr, wr, dx)
        return (dx.to(ctx.x_dtype) if need_dx else None, dw.to(ctx.w_dtype) if need_dw else None)


class Int8Linear(torch.nn.Module):
    """``Y = X W`` with 8-bit integer products in the forward and backward passes.

    Args:
        in_features, out_features: sizes (1 .. 131071).
    """

    def __init__(self, in_features, out_features, device=None, dtype=torch.float32):
        super().__init__()
        if not (1 <= in_features <= MAX_INNER and 1 <= out_features <= MAX_INNER):
            raise ValueError(f"in_features and out_features must be in [1, {MAX_INNER}]")
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.weight = torch.nn.Parameter(torch.empty(in_features, out_features, device=device, dtype=dtype))
        bound = 1.0 / math.sqrt(in_features)
        with torch.no_grad():
            self.weight.uniform_(-bound, bound)
        self._frozen = None

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}"

    @torch.no_grad()
    def freeze(self):
        """Lays out the 8-bit weight for serving; returns self."""
        lib, lock = _shared_context(self.weight.device)
        with lock:
            held = lib.new_int8(self.out_features, self.in_features)
            lib.quantize_int8(_operand(self.weight.detach()), colwise=held)
        self._frozen = (held, self.weight._version)
        return self

    def unfreeze(self):
        self._frozen = None
        return self

    def forward(self, x):
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        if x.device != self.weight.device:
            raise ValueError(f"x is on {x.device}, the weight on {self.weight.device}")
        lead = x.shape[:-1]
        flat = x.reshape(-1, self.in_features)
        if torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad):
            if flat.shape[0] > MAX_INNER:
                raise ValueError(f"at most {MAX_INNER} tokens in a pass with gradients, got {flat.shape[0]}")
            y = _Int8LinearFn.apply(flat, self.weight)
        elif self._frozen is not None:
            y = self._serve(flat)
        else:
            y = _Int8LinearFn.apply(flat.detach(), self.weight.detach())
        return y.reshape(*lead, self.out_features)

    def _serve(self, x):
        held, version = self._frozen
        if version != self.weight._version or held.codes.device != self.weight.device:
            raise RuntimeError("the weight changed since freeze(); call freeze() or unfreeze()")
        rows = x.shape[0]
        if rows == 0:
            return torch.empty(0, self.out_features, dtype=torch.bfloat16, device=x.device)
        lib, lock = _shared_context(x.device)
        with lock:
            y = _output(rows, self.out_features, torch.bfloat16, x.device)
            lib.linear_int8(_operand(x), lib.new_int8(rows, self.in_features), held, y)
        return y
