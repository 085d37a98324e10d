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
instead of quantizing the weight each time, until ``unfreeze()``.  They raise once the weight has changed,
as far as torch counts its changes (``freeze`` says which it does not).

To capture a training pass into a CUDA graph, run it once on the capturing stream first and let no
graph of an earlier pass over the same leaves live on (torch's own rule: their gradients would be
gathered on that pass's stream).

in_features and out_features go up to 131071, the bound of the exact sum, and so do the tokens
of a pass that the weight gets a gradient from; other passes take any number.  There is no CPU path.
"""

import functools
import math

import torch

from . import INT8_SCRATCH, Int8Struct
from .linear import _shared_context

MAX_INNER = 131071


def _output(rows, cols, dtype, device):
    """rows x cols with rows that start on 16 bytes.  Not a view: autograd refuses in-place changes of a
    view that a Function returns."""
    size = 8 if dtype == torch.bfloat16 else 4
    return torch.empty_strided((rows, cols), (-(-cols // size) * size, 1), dtype=dtype, device=device)


def _operand(M):
    """M as the quantizer reads it: fp32 or bf16, unit stride along a row."""
    if M.dtype not in (torch.float32, torch.bfloat16):
        M = M.float()
    rows, cols = M.shape
    if (M.stride(1) == 1 or cols == 1) and (M.stride(0) >= cols or rows == 1):
        return M
    return M.contiguous()     # transposed, or rows that are one and the same (an expanded gradient)


@functools.lru_cache(maxsize=256)
def _layout(sizes):
    """Bytes of one allocation for the operands of sizes (outer, inner, columns), and where each has its codes,
    scales and scratch in it.  columns: quantized column-wise, so with the scratch for that; the
    scratches lie side by side, so that one fill clears them."""
    at, places = 0, []
    for outer, inner, columns in sizes:
        ld = -(-inner // 16) * 16
        places.append((at, at + outer * ld, ld))
        at = -(-(at + outer * (ld + 4)) // 256) * 256
    out = []
    for (outer, inner, columns), (codes, scales, ld) in zip(sizes, places):
        out.append((outer, inner, ld, codes, scales, at if columns else None))
        at += 4 * outer * INT8_SCRATCH if columns else 0
    return at, out


def _buffers(device, sizes):
    """One allocation for the operands of sizes (outer, inner, columns), and their Int8Struct."""
    total, places = _layout(sizes)
    buf = torch.empty(total, dtype=torch.uint8, device=device)
    base = buf.data_ptr()
    return buf, [Int8Struct(base + codes, base + scales, outer, inner, ld, None if scratch is None else base + scratch)
                 for outer, inner, ld, codes, scales, scratch in places]


class _Int8LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        need_dx, need_dw = ctx.needs_input_grad
        rows, (m, n) = x.shape[0], weight.shape
        ctx.x_dtype, ctx.w_dtype, ctx.sizes = x.dtype, weight.dtype, (rows, m, n)
        if rows == 0:
            return torch.empty(0, n, dtype=torch.bfloat16, device=x.device)
        x, w = _operand(x), _operand(weight)
        # what the backward pass reads is kept, the rest goes with this call
        sizes = (((m, rows, False),) if need_dw else ()) + (((m, n, False),) if need_dx else ())
        kept, saved = _buffers(x.device, sizes) if sizes else (None, [])
        work, (xr, wc, *scratch) = _buffers(x.device, ((rows, m, False), (n, m, True)) + (((m, 1, True),) if need_dw else ()))
        if need_dw:
            saved[0].scratch = scratch[0].scratch
        y = _output(rows, n, torch.bfloat16, x.device)
        lib, lock = _shared_context(x.device)
        with lock:
            lib.int8_linear_fwd(x, w, y, xr, wc, Xcol=saved[0] if need_dw else None, Wrow=saved[-1] if need_dx else None)
        if kept is not None:
            ctx.save_for_backward(kept)
            ctx.kept = sizes
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_dx, need_dw = ctx.needs_input_grad
        rows, m, n = ctx.sizes
        if rows == 0:
            return (torch.empty(0, m, dtype=ctx.x_dtype, device=dy.device) if need_dx else None,
                    torch.zeros(m, n, dtype=ctx.w_dtype, device=dy.device) if need_dw else None)
        kept, = ctx.saved_tensors
        base = kept.data_ptr()
        saved = [Int8Struct(base + codes, base + scales, outer, inner, ld, None)
                 for outer, inner, ld, codes, scales, _ in _layout(ctx.kept)[1]]
        dy = _operand(dy)
        work, new = _buffers(dy.device, (((n, rows, True),) if need_dw else ()) + (((rows, n, False),) if need_dx else ()))
        dx = _output(rows, m, torch.bfloat16 if ctx.x_dtype == torch.bfloat16 else torch.float32, dy.device) if need_dx else None
        dw = _output(m, n, torch.float32, dy.device) if need_dw else None
        lib, lock = _shared_context(dy.device)
        with lock:
            lib.int8_linear_bwd(dy, Drow=new[-1] if need_dx else None, Dcol=new[0] if need_dw else None,
                                Xcol=saved[0] if need_dw else None, Wrow=saved[-1] if need_dx else None, dX=dx, dW=dw)
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
        """Lays out the 8-bit weight for serving; returns self.

        A weight that was written, replaced, cast or moved since makes the next served call raise.  Writes
        that torch does not count are not seen -- through ``weight.data``, by a replayed graph, to a weight made
        in inference mode: call freeze() again after those.  The weight's memory is held until unfreeze()."""
        lib, lock = _shared_context(self.weight.device)
        with lock:
            held = lib.new_int8(self.out_features, self.in_features)
            lib.quantize_int8(_operand(self.weight.detach()), colwise=held)
        # with its memory held, no other tensor comes to lie at its address
        self._frozen = (held, self.weight, self.weight.detach(), self._weight_version())
        return self

    def _weight_version(self):
        return None if self.weight.is_inference() else self.weight._version

    def _frozen_holds(self):
        """Whether the weight is the one that was laid out, by its identity, place, type and version."""
        _, weight, seen, version = self._frozen
        w = self.weight
        return (w is weight and w.data_ptr() == seen.data_ptr() and w.dtype is seen.dtype and w.device == seen.device and
                w.stride() == seen.stride() and self._weight_version() == version)

    def __getstate__(self):
        return dict(self.__dict__, _frozen=None)     # a copy lays its weight out itself

    def unfreeze(self):
        self._frozen = None
        return self

    def forward(self, x):
        weight = self.weight
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        if x.device != weight.device:
            raise ValueError(f"x is on {x.device}, the weight on {weight.device}")
        flat = x if x.dim() == 2 else x.reshape(-1, self.in_features)
        if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad):
            if weight.requires_grad and flat.shape[0] > MAX_INNER:     # dW contracts the tokens
                raise ValueError(f"at most {MAX_INNER} tokens in a pass with a gradient of the weight, got {flat.shape[0]}")
            y = _Int8LinearFn.apply(flat, weight)
        elif self._frozen is not None:
            y = self._serve(flat)
        else:
            y = _Int8LinearFn.apply(flat.detach(), weight.detach())
        return y if x.dim() == 2 else y.reshape(*x.shape[:-1], self.out_features)

    def _serve(self, x):
        held = self._frozen[0]
        if not self._frozen_holds():
            raise RuntimeError("the weight changed since freeze(); call freeze() or unfreeze()")
        rows = x.shape[0]
        if rows == 0:
            return torch.empty(0, self.out_features, dtype=torch.bfloat16, device=x.device)
        lib, lock = _shared_context(x.device)
        with lock:
            y = _output(rows, self.out_features, torch.bfloat16, x.device)
            lib.linear_int8(_operand(x), lib.new_int8(rows, self.in_features), held, y)
        return y
