"""AdamW for the master weights of the layers, one kernel launch for many tensors.

``AdamW`` is a ``torch.optim.Optimizer`` whose step runs in libmetis (metis_adamw_step):

    m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
    p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)

with the moments in fp32 (``state_bits=32``) or in one byte each (``state_bits=8``: small
floats that share an exponent byte among 128 consecutive elements).  Parameters are fp32 or
bf16, with gradients of the same type.  ``rounding="sr"`` rounds 8-bit moments and bf16
parameters stochastically (from ``seed``, the parameter's place in the optimizer and the
step, so a repeated run gives the same bits), ``"rn"`` to nearest.  Small changes against
the stored value -- a second moment with beta2 near 1, a bf16 weight with a small step -- are
lost on average by the nearest rounding and kept by the stochastic one.

``state_bits``, ``rounding``, ``lr``, ``betas``, ``eps`` and ``weight_decay`` may be set for each
parameter group.  With ``capturable=True`` the step count of a group lives on the device
(one for all its parameters) and ``lr`` may be a one-element fp32 CUDA tensor, so that step() can be
captured into a CUDA graph and replayed; take one step before the capture, which creates
the states.  There is no CPU path.
"""

import numpy as np
import torch

from . import OUT_BF16, OUT_F32
from .linear import _shared_context

BLOCK = 128    # elements that share an exponent of an 8-bit state

_ENTRY = np.dtype([("p", "u8"), ("g", "u8"), ("m", "u8"), ("v", "u8"), ("m_exponent", "u8"), ("v_exponent", "u8"),
                   ("n", "i8"), ("dtype", "i4"), ("id", "u4")])


def _dense_layout(t):
    """Whether the elements of t fill one stretch of memory, in whatever order of dimensions."""
    if t.is_contiguous():
        return True
    expected = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz > 1):
        if stride != expected:
            return False
        expected *= size
    return True


class AdamW(torch.optim.Optimizer):
    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32, rounding="sr",
                 seed=0, capturable=False):
        self.seed = int(seed)
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      rounding=rounding, capturable=capturable))

    def add_param_group(self, group):
        super().add_param_group(group)
        group = self.param_groups[-1]
        try:
            self._check_group(group)
        except ValueError:
            self.param_groups.pop()
            raise

    @staticmethod
    def _check_group(group):
        b1, b2 = group["betas"]
        if not (0.0 <= b1 < 1.0 and 0.0 <= b2 < 1.0):
            raise ValueError("betas must be in [0, 1)")
        if group["state_bits"] not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if group["rounding"] not in ("sr", "rn"):
            raise ValueError("rounding must be 'sr' or 'rn'")
        if not group["eps"] >= 0.0 or not group["weight_decay"] >= 0.0:
            raise ValueError("eps and weight_decay must not be negative")
        lr = group["lr"]
        if isinstance(lr, torch.Tensor):
            if not group["capturable"] or lr.numel() != 1 or lr.dtype != torch.float32 or not lr.is_cuda:
                raise ValueError("a tensor lr must be one fp32 element on the GPU, with capturable=True")
        elif not lr >= 0.0:
            raise ValueError("lr must not be negative")
        if len({id(p) for p in group["params"]}) != len(group["params"]):
            raise ValueError("a parameter appears twice in the group")
        for p in group["params"]:
            if p.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError(f"parameters must be fp32 or bf16, got {p.dtype}")
            if not _dense_layout(p):
                raise ValueError("a parameter's elements must fill one stretch of memory")

    # -- checkpoints -------------------------------------------------------------------
    def load_state_dict(self, state_dict):
        """As torch's, but every state keeps its own type (bytes stay bytes)."""
        super().load_state_dict(state_dict)
        flat = [p for group in self.param_groups for p in group["params"]]
        keys = [k for group in state_dict["param_groups"] for k in group["params"]]
        for p, key in zip(flat, keys):
            for name, value in state_dict["state"].get(key, {}).items():
                if isinstance(value, torch.Tensor):
                    self.state[p][name] = value.detach().to(device=p.device, copy=True)
                else:
                    self.state[p][name] = value
        for group in self.param_groups:
            if isinstance(group.get("step_count"), torch.Tensor) and group["params"]:
                group["step_count"] = group["step_count"].to(device=group["params"][0].device, copy=True)

    # -- the step ----------------------------------------------------------------------
    def _new_state(self, p, bits):
        state = {"step": 0}
        if bits == 32:
            state["exp_avg"] = torch.zeros_like(p, dtype=torch.float32, memory_format=torch.preserve_format)
            state["exp_avg_sq"] = torch.zeros_like(p, dtype=torch.float32, memory_format=torch.preserve_format)
        else:
            blocks = -(-p.numel() // BLOCK)
            for name in ("exp_avg", "exp_avg_sq"):
                state[name] = torch.zeros_like(p, dtype=torch.uint8, memory_format=torch.preserve_format)
                state[name + "_exponent"] = torch.zeros(blocks, dtype=torch.uint8, device=p.device)
        return state

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        first = 0
        for group in self.param_groups:
            self._step_group(group, first)
            first += len(group["params"])
        return loss

    def _step_group(self, group, first):
        bits, capturable = group["state_bits"], group["capturable"]
        calls = {}      # (device, step) -> rows of entries
        keep = []       # gradients copied into their parameter's layout
        todo = [(i, p, p.grad) for i, p in enumerate(group["params"]) if p.grad is not None]
        if not todo:
            return
        if not all(p.is_cuda for _, p, _ in todo):
            raise ValueError("parameters must be on a CUDA device")
        capturing = torch.cuda.is_current_stream_capturing()
        if capturing and not capturable:
            raise RuntimeError("step() under capture needs capturable=True")
        for i, p, g in todo:
            if g.layout != torch.strided or g.dtype != p.dtype or g.device != p.device:
                raise ValueError("a gradient must be dense, of its parameter's type and on its device")
            if not _dense_layout(p):
                raise ValueError("a parameter's elements must fill one stretch of memory")
            if g.stride() != p.stride():
                g = torch.empty_like(p, memory_format=torch.preserve_format).copy_(g)
                keep.append(g)
            state = self.state[p]
            if "exp_avg" not in state:
                if capturing:
                    raise RuntimeError("take one step before the capture: it creates the states")
                state.update(self._new_state(p, bits))
            m, v = state["exp_avg"], state["exp_avg_sq"]
            want = torch.uint8 if bits == 8 else torch.float32
            if m.dtype != want or v.dtype != want or m.shape != p.shape or v.shape != p.shape or \
                    m.stride() != p.stride() or v.stride() != p.stride():
                raise ValueError(f"a state does not fit its parameter with state_bits={bits}")
            me = ve = 0
            if bits == 8:
                e, f = state["exp_avg_exponent"], state["exp_avg_sq_exponent"]
                blocks = -(-p.numel() // BLOCK)
                if e.dtype != want or f.dtype != want or e.numel() != blocks or f.numel() != blocks or \
                        not e.is_contiguous() or not f.is_contiguous():
                    raise ValueError("a state's exponents do not fit its parameter")
                me, ve = e.data_ptr(), f.data_ptr()
            t = None
            if not capturable:
                t = state["step"] = int(state["step"]) + 1
            calls.setdefault((p.device, t), []).append(
                (p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), me, ve, p.numel(),
                 OUT_F32 if p.dtype == torch.float32 else OUT_BF16, first + i))
        if capturable:
            if len(calls) > 1:
                raise ValueError("the parameters of a capturable group must be on one device")
            (device, _), = calls
            count = group.get("step_count")
            if count is None:
                if capturing:
                    raise RuntimeError("take one step before the capture: it creates the states")
                count = group["step_count"] = torch.zeros((), dtype=torch.int64, device=device)
            count += 1
        lr, (b1, b2) = group["lr"], group["betas"]
        on_device = isinstance(lr, torch.Tensor)
        for (device, t), rows in calls.items():
            entries = np.array(rows, dtype=_ENTRY)
            lib, lock = _shared_context(device)
            with lock:
                lib.adamw_step(entries.ctypes.data, len(rows), 0.0 if on_device else float(lr), b1, b2, group["eps"],
                               group["weight_decay"], t or 1, bits, 1 if group["rounding"] == "sr" else 0, self.seed,
                               lr_dev=lr if on_device else None, step_dev=group["step_count"] if capturable else None)
