"""AdamW over a list of tensors: the handle that keeps the states and calls dflash2_adamw.

    opt = AdamW(params, grads, lr=1e-3, weight_decay=0.01, state_bits=8, master_weights=True)
    opt.step(grad_scale=clip)      # one launch for up to 320 tensors, nothing uploaded
"""
from __future__ import annotations

from operator import is_

import torch

import dflash2_draft_block_gb300 as _pkg

from . import _abi

ADAMW_BLOCK = 256
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_NAMES = {32: ("exp_avg", "exp_avg_sq"),
          8: ("exp_avg", "exp_avg_rms", "exp_avg_scale", "exp_avg_rms_scale")}


def _each(value, n, name):
    """A number for every tensor, or one number a tensor."""
    if isinstance(value, (int, float)):
        return [float(value)] * n
    value = [float(v) for v in value]
    if len(value) != n:
        raise ValueError(f"{name} must be one number or {n} of them, got {len(value)}")
    return value


def _tensor(t, name, dtypes, numel, device):
    if not isinstance(t, torch.Tensor) or not _pkg._on_device(t):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got shape {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the parameters on {device}")
    return t


class AdamW:
    """AdamW (decoupled weight decay) over `params`, CUDA tensors in bf16 or fp32.

    grads           one tensor a parameter, read at every step; None: each step's `grads`,
                    or the parameters' .grad (a parameter without one is left out)
    lr, weight_decay   numbers, or one a parameter
    state_bits      32: exp_avg and exp_avg_sq in fp32.  8: exp_avg and exp_avg_rms, the
                    root of the second moment, as torch.float8_e4m3fn in units of one fp32
                    scale per 256 elements (exp_avg_scale, exp_avg_rms_scale): element i
                    stands for value[i].float() * scale[i // 256]
    master_weights  True: an fp32 copy of every parameter is kept, updated and rounded into
                    it; or the list of those copies
    state, step     the lists named above and the steps done, as state_dict() gives them;
                    None and 0: zeros

    The states belong to the stream the handle was made on; `step` runs on `stream` (default:
    the current one), and the caller orders the streams where they differ."""

    def __init__(self, params, grads=None, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                 state_bits=32, master_weights=None, state=None, step=0):
        if state_bits not in _NAMES:
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        self.params = list(params)
        n = len(self.params)
        self.state_bits, self.step_count, self.eps = state_bits, int(step), float(eps)
        self.beta1, self.beta2 = (float(b) for b in betas)
        self.lr, self.weight_decay = _each(lr, n, "lr"), _each(weight_decay, n, "weight_decay")
        self.device = self.params[0].device if n else None
        for i, p in enumerate(self.params):
            _tensor(p, f"params[{i}]", _DTYPES, None, self.device)
        if n:
            _pkg._device(self.params[0])
        if master_weights is True:
            master_weights = [p.detach().to(torch.float32, copy=True) for p in self.params]
        self.master_weights = list(master_weights) if master_weights else None
        if self.master_weights is not None:
            self._list(self.master_weights, "master_weights", torch.float32, 1)
        self.state = self._fresh() if state is None else {k: list(state[k]) for k in _NAMES[state_bits]}
        for name, ts in self.state.items():
            scale = name.endswith("_scale")
            held = torch.float8_e4m3fn if state_bits == 8 and not scale else torch.float32
            self._list(ts, name, held, ADAMW_BLOCK if scale else 1)
        self.grads = list(grads) if grads is not None else None
        self._bound = self._ptrs = self._table = None

    def _list(self, ts, name, dtype, per):
        if len(ts) != len(self.params):
            raise ValueError(f"{name} must hold one tensor a parameter")
        for i, (t, p) in enumerate(zip(ts, self.params)):
            _tensor(t, f"{name}[{i}]", (dtype,), -(-p.numel() // per), self.device)

    def _fresh(self):
        """Zero states: one allocation a kind, each tensor's part on a block of its own."""
        blocks = [-(-p.numel() // ADAMW_BLOCK) for p in self.params]
        state = {}
        for name in _NAMES[self.state_bits]:
            scale = name.endswith("_scale")
            per = 1 if scale else ADAMW_BLOCK
            flat = torch.zeros(sum(blocks) * per, device=self.device,
                               dtype=torch.uint8 if self.state_bits == 8 and not scale else torch.float32)
            if flat.dtype == torch.uint8:
                flat = flat.view(torch.float8_e4m3fn)
            at, parts = 0, []
            for b, p in zip(blocks, self.params):
                parts.append(flat[at:at + (b if scale else p.numel())])
                at += b * per
            state[name] = parts
        return state

    def _bind(self, grads):
        """The descriptors of a step whose tensors are not those of the last one."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        if self.params:
            _pkg._device(self.params[0])
        table = (_abi.AdamWTensor * len(self.params))()
        first, second = _NAMES[self.state_bits][:2]
        for i, (p, g) in enumerate(zip(self.params, grads)):
            e = table[i]
            e.lr, e.weight_decay = self.lr[i], self.weight_decay[i]
            e.param_dtype = _DTYPES[_tensor(p, f"params[{i}]", _DTYPES, self.state[first][i].numel(), self.device).dtype]
            if g is None:
                continue  # n = 0: left out
            e.grad_dtype = _DTYPES[_tensor(g, f"grads[{i}]", _DTYPES, p.numel(), self.device).dtype]
            e.param, e.grad, e.n = p.data_ptr(), g.data_ptr(), p.numel()
            e.exp_avg, e.exp_avg_2 = self.state[first][i].data_ptr(), self.state[second][i].data_ptr()
            if self.master_weights is not None:
                e.master = self.master_weights[i].data_ptr()
            if self.state_bits == 8:
                e.exp_avg_scale = self.state["exp_avg_scale"][i].data_ptr()
                e.exp_avg_2_scale = self.state["exp_avg_rms_scale"][i].data_ptr()
        return table

    def step(self, grads=None, *, grad_scale=None, lr=None, stream=None):
        """One step.  grad_scale: an fp32 CUDA scalar the gradients are multiplied by (a NaN
        or infinite one leaves the tensors and states as they are; the step counts all the
        same, as the host does not wait to see).  lr: new learning rates."""
        if grads is None:
            grads = self.grads if self.grads is not None else [p.grad for p in self.params]
        if grad_scale is not None:
            _tensor(grad_scale, "grad_scale", (torch.float32,), 1, self.device)
        if lr is not None:
            self.lr = _each(lr, len(self.params), "lr")
            self._bound = None
        # the same tensors where they were: the last step's descriptors hold
        ptrs = [t.data_ptr() for t in self.params] + [0 if g is None else g.data_ptr() for g in grads]
        if self._bound is None or ptrs != self._ptrs or len(grads) != len(self._bound) or \
                not all(map(is_, grads, self._bound)):
            self._bound = None
            self._table = self._bind(grads)
            self._ptrs, self._bound = ptrs, list(grads)
        if not self.params:
            return
        rc = _pkg.lib().dflash2_adamw(self._table, len(self.params), self.state_bits, self.beta1, self.beta2,
                                      self.eps, self.step_count + 1, _pkg._ptr(grad_scale),
                                      _pkg._stream(stream, self.device))
        _pkg._check("dflash2_adamw", rc)
        self.step_count += 1

    def state_dict(self):
        """The states (not copies), the master weights and the steps done."""
        return {"state": self.state, "step": self.step_count, "master_weights": self.master_weights}
