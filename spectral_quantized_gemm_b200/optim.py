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
(one for all its parameters; it goes on from theirs, and theirs from it, where a group's
``capturable`` is changed between steps) and ``lr`` may be a one-element fp32 CUDA tensor, so that step() can be
captured into a CUDA graph and replayed; take one step before the capture, which creates
the states.  There is no CPU path.
"""

import array
import itertools
import operator

import torch

from . import OUT_BF16, OUT_F32
from .linear import _shared_context

BLOCK = 128    # elements that share an exponent of an 8-bit state

ENTRY_WORDS = 8    # 64-bit words of a metis_adamw_tensor: six addresses, n, dtype | id << 32


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


_address, _numel, _contiguous = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous
_grad, _dtype, _on_gpu = operator.attrgetter("grad"), operator.attrgetter("dtype"), operator.attrgetter("is_cuda")
_step = operator.itemgetter("step")
# The parameters are written behind torch's back; whoever compares versions (autograd's check of saved
# tensors, a frozen layer) learns of it here.
_increment_version = torch.autograd.graph.increment_version


class _Plan:
    """The entries of a group's last step and the objects that they were made from.  The next step
    uses them again, with the addresses of its gradients, if every object is still the same and
    lies where it lay; anything else goes through the checks of a first step."""

    def __init__(self, params, dtypes, sizes, tensors, all_states, states, entries, device):
        self.params, self.dtypes, self.sizes, self.tensors = params, dtypes, sizes, tensors
        self.all_states, self.states, self.entries, self.device = all_states, states, entries, device
        self.where = self.addresses()

    def addresses(self):
        return list(map(_address, self.tensors))

    def renew(self, params, all_states, keys, t):
        """Whether the plan holds for states of t steps (None: not counted there); then its entries are up to date."""
        if len(params) != len(self.params) or not all(map(operator.is_, params, self.params)) or \
                len(all_states) != len(self.all_states) or not all(map(operator.is_, all_states.values(), self.all_states)):
            return False
        grads = list(map(_grad, params))
        if any(map(operator.is_, grads, itertools.repeat(None))) or list(map(_dtype, grads)) != self.dtypes or \
                list(map(_numel, grads)) != self.sizes or not all(map(_contiguous, grads)) or not all(map(_on_gpu, grads)):
            return False
        now = itertools.chain.from_iterable(map(operator.itemgetter(k), self.states) for k in keys)
        if not all(map(operator.is_, self.tensors[len(params):], now)) or self.addresses() != self.where:
            return False
        if t is not None:
            if list(map(_step, self.states)).count(t) != len(params):
                return False
        self.entries[1::ENTRY_WORDS] = array.array("Q", map(_address, grads))
        return True


_KEYS = {32: ("exp_avg", "exp_avg_sq"), 8: ("exp_avg", "exp_avg_sq", "exp_avg_exponent", "exp_avg_sq_exponent")}


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
            for name in ("step_count", "lr"):
                if isinstance(group.get(name), torch.Tensor) and group["params"]:
                    group[name] = group[name].to(device=group["params"][0].device, copy=True)

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
        plans = self.__dict__.setdefault("_plans", {})
        if len(plans) > len(self.param_groups):                 # groups have gone or changed their options
            plans.clear()
        first = 0
        for number, group in enumerate(self.param_groups):
            plan = plans.get((number, first, group["state_bits"], group["capturable"]))
            if plan is None or not self._step_again(group, plan):
                plans[number, first, group["state_bits"], group["capturable"]] = self._step_group(group, first)
            first += len(group["params"])
        return loss

    def __getstate__(self):
        return dict(super().__getstate__(), seed=self.seed)     # the plans stay behind

    def _step_again(self, group, plan):
        """The step from a plan that still holds; False if it does not."""
        if torch.cuda.is_current_stream_capturing() and not group["capturable"]:
            return False
        if group["capturable"] != (group.get("step_count") is not None):     # changed since: the counts move first
            return False
        t = None if group["capturable"] else plan.states[0]["step"]
        if not plan.renew(group["params"], self.state, _KEYS[group["state_bits"]], t):
            return False
        self._launch(group, plan.device, t, plan.entries)
        if t is not None:
            for state in plan.states:
                state["step"] = t + 1
        _increment_version(plan.params)
        return True

    def _launch(self, group, device, t, rows):
        """One call for the entries of a device; t: their steps so far, or None for the group's count."""
        lr, (b1, b2) = group["lr"], group["betas"]
        on_device = isinstance(lr, torch.Tensor)
        lib, lock = _shared_context(device)
        count = group["step_count"] if t is None else None
        if count is not None:
            count += 1
        try:
            with lock:
                lib.adamw_step(rows.buffer_info()[0], len(rows) // ENTRY_WORDS, 0.0 if on_device else float(lr), b1, b2,
                               group["eps"], group["weight_decay"], 1 if t is None else t + 1, group["state_bits"],
                               1 if group["rounding"] == "sr" else 0, self.seed, lr_dev=lr if on_device else None,
                               step_dev=count)
        except Exception:
            if count is not None:
                count -= 1                                       # a step that was refused does not count
            raise

    def _step_group(self, group, first):
        bits, capturable = group["state_bits"], group["capturable"]
        todo = [(i, p, g) for i, p in enumerate(group["params"]) if (g := p.grad) is not None]
        if not todo:
            return None
        device = todo[0][1].device
        if device.type != "cuda":
            raise ValueError("parameters must be on a CUDA device")
        capturing = torch.cuda.is_current_stream_capturing()
        if capturing and not capturable:
            raise RuntimeError("step() under capture needs capturable=True")
        calls = {}      # (device, steps taken) -> flat list of the entries' numbers
        keep = []       # gradients copied into their parameter's layout
        counted = []    # (state, its next step), set once all is launched
        state_dtype = torch.uint8 if bits == 8 else torch.float32
        states = self.state
        t, fresh = None, 0
        if not capturable and (count := group.pop("step_count", None)) is not None:
            for p in group["params"]:                            # the group was capturable until now
                if p in states:
                    states[p]["step"] = int(count)
        for i, p, g in todo:
            dtype, n = p.dtype, p.numel()
            if not (g.layout is torch.strided and g.dtype is dtype and g.numel() == n and p.device == g.device and p.is_cuda):
                raise ValueError("a gradient must be dense, of its parameter's type and size, both on one CUDA device")
            plain = p.is_contiguous()
            if not (plain and g.is_contiguous()):
                g = self._same_layout(p, g, keep)
            state = states[p]
            if "exp_avg" not in state:
                if capturing:
                    raise RuntimeError("take one step before the capture: it creates the states")
                state.update(self._new_state(p, bits))
                fresh += 1
            m, v = state["exp_avg"], state["exp_avg_sq"]
            if not (m.dtype is state_dtype and v.dtype is state_dtype and m.numel() == n and v.numel() == n and
                    m.device == v.device == p.device and
                    (m.is_contiguous() and v.is_contiguous() if plain else m.stride() == p.stride() == v.stride())):
                raise ValueError(f"a state does not fit its parameter with state_bits={bits}")
            e, f = m, v
            if bits == 8:
                e, f = state["exp_avg_exponent"], state["exp_avg_sq_exponent"]
                blocks = -(-n // BLOCK)
                if not (e.dtype is state_dtype and f.dtype is state_dtype and e.numel() == blocks and f.numel() == blocks and
                        e.is_contiguous() and f.is_contiguous() and e.device == f.device == p.device):
                    raise ValueError("a state's exponents do not fit its parameter")
            if not capturable:
                t = int(state["step"])
                counted.append((state, t + 1))
            rows = calls.get((p.device, t))
            if rows is None:
                rows = calls[p.device, t] = array.array("Q")
            # the last word holds the struct's two 32-bit fields, dtype and id
            rows.extend((p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), e.data_ptr(), f.data_ptr(), n,
                         (OUT_F32 if dtype is torch.float32 else OUT_BF16) | (first + i) << 32))
        taken = [p.data_ptr() for _, p, _ in todo if p.numel()]
        if len(set(taken)) < len(taken):
            raise ValueError("two parameters of a group lie at the same address")
        if capturable:
            if len(calls) > 1:
                raise ValueError("the parameters of a capturable group must be on one device")
            count = group.get("step_count")
            if count is None:
                if capturing:
                    raise RuntimeError("take one step before the capture: it creates the states")
                steps = {int(states[p].get("step", 0)) for p in group["params"] if p in states} - {0}
                if len(steps) > 1:
                    raise ValueError("the parameters of a capturable group must have taken the same number of steps")
                count = group["step_count"] = torch.full((), max(steps, default=0), dtype=torch.int64, device=device)
            elif fresh and fresh == sum("exp_avg" in states[p] for p in group["params"] if p in states):
                count.zero_()                                    # no state has seen a step of it
        for (device, t), rows in calls.items():
            self._launch(group, device, t, rows)
        for state, step in counted:
            state["step"] = step
        _increment_version([p for _, p, _ in todo])
        # a plan for the next step where this one was regular
        if len(calls) > 1 or keep or len(todo) != len(group["params"]) or not all(p.is_contiguous() for _, p, _ in todo):
            return None
        params, own = [p for _, p, _ in todo], [states[p] for _, p, _ in todo]
        return _Plan(params, [p.dtype for p in params], [p.numel() for p in params],
                     params + [s[k] for k in _KEYS[bits] for s in own], list(states.values()), own, rows, device)

    @staticmethod
    def _same_layout(p, g, keep):
        """The gradient in the order of the parameter's memory; a copy is put into `keep`."""
        if not _dense_layout(p):
            raise ValueError("a parameter's elements must fill one stretch of memory")
        if g.shape != p.shape:
            raise ValueError("a gradient must have its parameter's shape")
        if g.stride() != p.stride():
            g = torch.empty_like(p, memory_format=torch.preserve_format).copy_(g)
            keep.append(g)
        return g
