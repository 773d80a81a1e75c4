"""AdamW over a list of tensors: the handle that keeps the states and calls dflash2_adamw.

    opt = AdamW(params, grads, lr=1e-3, weight_decay=0.01, state_bits=8, master_weights=True)
    opt.step(grad_scale=clip)      # one launch for up to 320 tensors, nothing uploaded
"""
from __future__ import annotations

import ctypes as ct
from array import array

import torch
from torch.autograd.graph import increment_version

import dflash2_draft_block_gb300 as _pkg

from . import _abi

ADAMW_BLOCK = 256
_F32 = (torch.float32,)
_UNSUPPORTED = 2  # DF2_ERR_UNSUPPORTED
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_NAMES = {32: ("exp_avg", "exp_avg_sq"),
          8: ("exp_avg", "exp_avg_rms", "exp_avg_scale", "exp_avg_rms_scale")}
_FIELDS = ("param", "exp_avg", "exp_avg_2", "exp_avg_scale", "exp_avg_2_scale")  # of params, then _NAMES
_WORDS = ct.sizeof(_abi.AdamWTensor) // 8  # of 64 bits, in a descriptor

# (by map() a list's worth takes two thirds of the time of a loop)
_PTR, _NUMEL, _DENSE, _DEVICE = (getattr(torch.Tensor, k) for k in ("data_ptr", "numel", "is_contiguous", "get_device"))


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
                    or the parameters' .grad.  A parameter without one is left out, and the step
                    is none of its own: its bias corrections count the steps it took
    lr, weight_decay   numbers, or one a parameter
    state_bits      32: exp_avg and exp_avg_sq in fp32.  8: exp_avg and exp_avg_rms, the
                    root of the second moment, as torch.float8_e4m3fn in units of one fp32
                    scale per 256 elements (exp_avg_scale, exp_avg_rms_scale): element i
                    stands for value[i].float() * scale[i // 256]
    master_weights  True: an fp32 copy of every parameter is kept, updated and rounded into
                    it; or the list of those copies
    state, step     the lists named above and the steps done (one number, or one a
                    parameter), as state_dict() gives them; None and 0: zeros

    Every step uses params, grads, master_weights, state, lr, weight_decay and the other
    attributes as they are then: tensors may move, and be replaced by others of their
    type and length.  Between steps the handle keeps no gradient that it was not made with.

    The states belong to the stream the handle was made on; `step` runs on `stream` (default:
    the current one), and the caller orders the streams where they differ, and keeps the
    gradients until such a step has read them."""

    def __init__(self, params, grads=None, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                 state_bits=32, master_weights=None, state=None, step=0):
        if state_bits not in _NAMES:
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        self.params = list(params)
        n = len(self.params)
        self.state_bits, self.eps = state_bits, float(eps)
        steps = [int(t) for t in step] if isinstance(step, (list, tuple)) else [int(step)] * max(n, 1)
        if len(steps) != max(n, 1):
            raise ValueError(f"step must be one number or {n} of them, got {len(steps)}")
        self.step_count = max(steps)
        # how many of them each parameter was left out of (None: none of any)
        self._late = [self.step_count - t for t in steps] if len(set(steps)) > 1 else None
        self.beta1, self.beta2 = (float(b) for b in betas)
        self.lr, self.weight_decay = _each(lr, n, "lr"), _each(weight_decay, n, "weight_decay")
        self.device = self.params[0].device if n else None
        self._cuda = self.device.index if n and self.device.type == "cuda" else None
        for i, p in enumerate(self.params):
            _tensor(p, f"params[{i}]", _DTYPES, None, self.device)
        if n:
            _pkg._device(self.params[0])
        if master_weights is True:
            master_weights = [p.detach().to(torch.float32, copy=True) for p in self.params]
        self.master_weights = list(master_weights) if master_weights else None
        self.state = self._fresh() if state is None else {k: list(state[k]) for k in _NAMES[state_bits]}
        self._check()
        self.grads = list(grads) if grads is not None else None
        self._table = self._words = self._seen = self._rates = None

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

    def _check(self):
        """Parameters, masters and states that fit one another and the device."""
        for i, p in enumerate(self.params):
            _tensor(p, f"params[{i}]", _DTYPES, None, self.device)
        if self.master_weights is not None:
            self._list(self.master_weights, "master_weights", torch.float32, 1)
        for name in _NAMES[self.state_bits]:
            scale = name.endswith("_scale")
            held = torch.float8_e4m3fn if self.state_bits == 8 and not scale else torch.float32
            self._list(self.state[name], name, held, ADAMW_BLOCK if scale else 1)

    def _column(self, field, values, code="Q"):
        """A field of every descriptor."""
        self._words[code][getattr(_abi.AdamWTensor, field).offset // 8::_WORDS] = array(code, values)

    def _describe(self, grads):
        """The step's descriptors, from the tensors and rates as they are now.  Every tensor's
        address and bytes and a gradient's type and layout are read at every step, and nothing
        is kept but those; where they are what they were, the checks and the columns hold.
        Returns whether every parameter has a gradient."""
        params, n = self.params, len(self.params)
        if len(grads) != n:
            raise ValueError(f"{len(grads)} gradients for {n} parameters")
        if n == 0:
            return True
        if self._table is None:
            words = array("Q", bytes(8 * _WORDS * n))
            self._table = (_abi.AdamWTensor * n).from_buffer(words)
            self._words = {"Q": memoryview(words), "d": memoryview(words).cast("B").cast("d")}
        if n != len(self._table):
            raise ValueError(f"the handle was made for {len(self._table)} parameters, now there are {n}")
        given, missing = grads, [i for i, g in enumerate(grads) if g is None]
        if missing:  # their parameters stand in, and their lengths become 0
            given = [p if g is None else g for p, g in zip(params, grads)]
        every = [*given, *params]
        for name in _NAMES[self.state_bits]:
            every += self.state[name]
        if self.master_weights is not None:
            every += self.master_weights
        seen = list(map(_PTR, every)), [t.nbytes for t in every], [g.dtype for g in given], missing
        if seen != self._seen or not all(map(_DENSE, given)):
            last, self._seen = self._seen, None
            if last is None or any(a[n:] != b[n:] for a, b in zip(seen[:2], last)):
                self._held(seen[0])
            if list(map(_NUMEL, given)) != self._numels or not all(map(_DENSE, given)) or \
                    not _DTYPES.keys() >= set(seen[2]) or set(map(_DEVICE, given)) != self._index:
                for i, (p, g) in enumerate(zip(params, given)):
                    _tensor(g, f"grads[{i}]", _DTYPES, p.numel(), self.device)
            self._column("grad", seen[0][:n])
            self._column("n", [0 if g is None else k for g, k in zip(grads, self._numels)])
            # and grad_dtype, the other half of the word
            self._column("param_dtype", [p | _DTYPES[d] << 32 for p, d in zip(self._codes, seen[2])])
            self._seen = seen

        if (self.lr, self.weight_decay) != self._rates:
            self.lr, self.weight_decay = _each(self.lr, n, "lr"), _each(self.weight_decay, n, "weight_decay")
            self._column("lr", self.lr, "d")
            self._column("weight_decay", self.weight_decay, "d")
            self._rates = list(self.lr), list(self.weight_decay)
        return not missing

    def _held(self, ptrs):
        """Checks and columns of the parameters, the states and the masters (ptrs: after the
        gradients', in this order)."""
        self._check()
        n = len(self.params)
        fields = _FIELDS[:1 + len(_NAMES[self.state_bits])]
        for i, field in enumerate(fields, 1):
            self._column(field, ptrs[i * n:(i + 1) * n])
        self._column("master", ptrs[(1 + len(fields)) * n:] or [0] * n)
        self._numels, self._codes = [p.numel() for p in self.params], [_DTYPES[p.dtype] for p in self.params]
        self._index = {p.get_device() for p in self.params}

    def step(self, grads=None, *, grad_scale=None, lr=None, stream=None):
        """One step.  grad_scale: an fp32 CUDA scalar the gradients are multiplied by (a NaN
        or infinite one leaves the tensors and states as they are; the step counts all the
        same, as the host does not wait to see).  lr: new learning rates.

        The step's number and rates are the host's, so a step is refused while its stream is
        being captured into a CUDA graph."""
        if grads is None:
            grads = self.grads if self.grads is not None else [p.grad for p in self.params]
        if grad_scale is not None:
            _tensor(grad_scale, "grad_scale", _F32, 1, self.device)
        if lr is not None:
            self.lr = _each(lr, len(self.params), "lr")
        whole = self._describe(grads)
        if not self.params:
            return
        if self._cuda is None or torch.cuda.current_device() != self._cuda:
            _pkg._device(self.params[0])  # refuses another device than the current one
        call = self.state_bits, self.beta1, self.beta2, self.eps
        on = _pkg._ptr(grad_scale), _pkg._stream(stream, self.device)
        late = self._late
        groups = (0,) if late is None else {k for k, g in zip(late, grads) if g is not None}
        for group in groups:  # of parameters at the same step of their own
            table = self._table
            if len(groups) > 1:
                table = type(table).from_buffer_copy(table)
                for e, k in zip(table, late):
                    e.n = e.n if k == group else 0
            rc = _pkg.lib().dflash2_adamw(table, len(table), *call, self.step_count + 1 - group, *on)
            if rc == _UNSUPPORTED and _pkg._capturing(stream, self.device):
                raise RuntimeError("an AdamW step cannot be captured: its replays would all be this step, with its "
                                   "bias corrections and rates")
            _pkg._check("dflash2_adamw", rc)
        # written behind autograd's back: a backward through weights saved before must notice
        increment_version(self.params if whole else [p for p, g in zip(self.params, grads) if g is not None])
        self.step_count += 1
        if not whole:
            self._late = [k + (g is None) for k, g in zip(late or [0] * len(grads), grads)]

    def state_dict(self):
        """The states (not copies), the master weights and the steps done (a list of each
        parameter's, once one was left out)."""
        steps = self.step_count if self._late is None else [self.step_count - k for k in self._late]
        return {"state": self.state, "step": steps, "master_weights": self.master_weights}
