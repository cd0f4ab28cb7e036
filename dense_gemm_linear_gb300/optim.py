"""AdamW over many torch CUDA tensors (dgl_adamw)."""
from __future__ import annotations

import ctypes

import torch

from . import ADAMW_BLOCK, OUT_F32, AdamWDesc, AdamWTensor, _check, load_library
from .head import _not_here, _packed
from .norm import _CODES

_F32 = torch.float32
_STATES = {32: (_F32, _F32), 8: (torch.float8_e4m3fn, torch.float8_e5m2)}


def _code(t, name, i):
    code = _CODES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise TypeError(f"{name}[{i}] must be a bf16 or fp32 CUDA tensor")
    return code


def _flat(t, name, i, device):
    """Checks a contiguous tensor on the current device; returns its address."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _not_here(t, f"{name}[{i}]", device)
    if not t.is_contiguous():
        raise ValueError(f"{name}[{i}] must be contiguous")
    return t.data_ptr()


def _apart(written):
    """Refuses memory that a step would write twice; written: (address, bytes, list, place) of all that it writes."""
    end, last = 0, None
    for at, size, name, i in sorted(written):
        if at < end and size:
            raise ValueError(f"{name}[{i}] and {last[0]}[{last[1]}] overlap: the updates would race")
        if size:
            end, last = at + size, (name, i)


def _unmoved(tensors, places, indexes):
    return [t.data_ptr() for t in tensors] == places


# (torch's own form of the same takes half the time: 3 us for 98 tensors)
_unmoved = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", _unmoved)


def _kept(name):
    """A list of tensors that the optimizer holds the memory of: handed out as aliases, replaced as a whole."""

    def get(self):
        held = self._held[name]
        return None if held is None else tuple(None if t is None else t.detach() for t in held)

    def replace(self, given):
        self._lay(**{name: given})

    return property(get, replace)


class AdamW:
    """AdamW (Adam with decoupled weight decay) over a list of tensors: a launch a step for each kind of
    them (types, with a master or not, in 16-byte units or not).

    params: bf16 or fp32 CUDA tensors, contiguous, updated in place.  grads: a
    gradient for each, bf16 or fp32, of the same shape: the buffers that every
    step reads unless it is given others (None: each step is given them).
    weight_decay: a number, or one for each tensor.  master: fp32 copies of bf16
    params, which are then updated, params becoming their roundings; True makes
    them from the params.  state_bits: 32, or 8 for E4M3 and E5M2 states with an
    fp32 scale for each 128 elements, rounded at random with `seed`.

    exp_avg, exp_avg_sq, in 8 bits also exp_avg_scale and exp_avg_sq_scale
    (sequences of 1-D tensors), and steps (int64 [1], the steps taken) are the state: made
    as zeros when None, kept as attributes of those names, and enough with the
    params and masters to go on from a checkpoint.  All tensors are on the
    device that is current, then and at every step.  What a step writes (params,
    masters, state) overlaps nothing else that it reads or writes.

    The optimizer holds the memory of its state and masters.  Their attributes are
    tuples of aliases, through which values can be read and changed; assigning a
    whole list (or steps, or grads) replaces the tensors, with the checks of the
    start.  Where a param or a gradient given at the start has moved since the
    last step (`p.data = ...`), all are checked again and its new memory is taken; the
    old is let go then.  A captured step keeps the addresses of its capture.
    """

    def __init__(self, params, grads=None, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, master=None,
                 state_bits=32, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None, steps=None,
                 seed=0):
        device = torch.cuda.current_device()
        params = list(params)
        n = len(params)
        for i, p in enumerate(params):
            _code(p, "params", i)
        if exp_avg is not None and len(exp_avg) and exp_avg[0].dtype != _F32:
            state_bits = 8
        if state_bits not in _STATES:
            raise ValueError("state_bits must be 8 or 32")
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(decay) != n:
            raise ValueError("weight_decay has one entry for each of params")
        if master is True:
            master = [p.detach().to(_F32, copy=True).contiguous() if p.dtype == torch.bfloat16 else None for p in params]
        self.device, self.state_bits, self.lr = device, state_bits, lr
        self._decay = decay
        sizes = [p.numel() for p in params]
        if state_bits == 8:
            blocks = [-(-k // ADAMW_BLOCK) for k in sizes]
            exp_avg_scale = self._zeros(blocks, _F32) if exp_avg_scale is None else exp_avg_scale
            exp_avg_sq_scale = self._zeros(blocks, _F32) if exp_avg_sq_scale is None else exp_avg_sq_scale
        m_type, v_type = _STATES[state_bits]
        self._ticket = torch.zeros(1, dtype=torch.int32, device=device)
        self._desc = AdamWDesc(None, self._ticket.data_ptr(), None, None, 0.0, betas[0], betas[1], eps,
                               seed & (2**64 - 1), state_bits)
        self._held = {}
        self._lay(params=params, grads=grads, master=master, exp_avg_scale=exp_avg_scale,
                  exp_avg_sq_scale=exp_avg_sq_scale, exp_avg=self._zeros(sizes, m_type) if exp_avg is None else exp_avg,
                  exp_avg_sq=self._zeros(sizes, v_type) if exp_avg_sq is None else exp_avg_sq,
                  steps=torch.zeros(1, dtype=torch.int64, device=device) if steps is None else steps)

    params = property(lambda self: tuple(self._held["params"]))
    master = _kept("master")
    exp_avg = _kept("exp_avg")
    exp_avg_sq = _kept("exp_avg_sq")
    exp_avg_scale = _kept("exp_avg_scale")
    exp_avg_sq_scale = _kept("exp_avg_sq_scale")

    @property
    def grads(self):
        grads = self._held["grads"]
        return None if grads is None else tuple(grads)

    @grads.setter
    def grads(self, grads):
        self._lay(grads=grads)

    @property
    def steps(self):
        return self._held["steps"].detach()

    @steps.setter
    def steps(self, steps):
        self._lay(steps=steps)

    def _zeros(self, sizes, dtype):
        """Tensors of a state, in one buffer, each in whole blocks of 128 elements."""
        slots = [-(-k // ADAMW_BLOCK) * ADAMW_BLOCK for k in sizes]
        whole = torch.zeros(sum(slots), dtype=torch.uint8 if dtype != _F32 else _F32, device=self.device).view(dtype)
        return [s[:k] for s, k in zip(whole.split(slots), sizes)] if slots else []

    def _lay(self, **given):
        """Checks all tensors, those given in place of the ones held, and lays out the table of the library's calls."""
        held = {**self._held, **given}
        params, master, device = list(held["params"]), held["master"], self.device
        if master is not None and len(master) != len(params):
            raise ValueError("master has one entry for each of params")
        table = (AdamWTensor * len(params))()
        sizes, written = [], []
        for i, (t, p, decay) in enumerate(zip(table, params, self._decay)):
            t.param_dtype = code = _code(p, "params", i)
            at, n = _flat(p, "params", i, device), p.numel()
            t.param, t.n, t.weight_decay = at, n, decay
            sizes.append(n)
            written.append((at, n * (4 if code == OUT_F32 else 2), "params", i))
            if master is not None and master[i] is not None:
                if code == OUT_F32:
                    raise TypeError(f"master[{i}] is given beside a param of fp32")
                t.master = at = _packed(master[i], f"master[{i}]", _F32, p.shape, device)
                written.append((at, n * 4, "master", i))
        blocks = [-(-k // ADAMW_BLOCK) for k in sizes]
        m_type, v_type = _STATES[self.state_bits]
        states = [("exp_avg", sizes, m_type), ("exp_avg_sq", sizes, v_type)]
        if self.state_bits == 8:
            states += [("exp_avg_scale", blocks, _F32), ("exp_avg_sq_scale", blocks, _F32)]
        elif held["exp_avg_scale"] is not None or held["exp_avg_sq_scale"] is not None:
            raise ValueError("states of 32 bits have no scales")
        for name, lengths, dtype in states:
            self._state(name, held[name], lengths, dtype, table, written)
        steps = _packed(held["steps"], "steps", torch.int64, (1,), device)
        _apart(written + [(steps, 8, "steps", 0), (self._ticket.data_ptr(), 4, "the ticket", 0)])
        grads = None if held["grads"] is None else list(held["grads"])
        if grads is not None:
            self._take(grads, table, params)
        # what is the optimizer's own is held by aliases, whose memory nothing but the optimizer lets go
        for name, _, _ in states:
            held[name] = [t.data for t in held[name]]
        held.update(params=params, grads=grads, steps=held["steps"].data,
                    master=None if master is None else [None if t is None else t.data for t in master])
        watched = params + (grads or [])
        self._held, self._table, self._desc.steps = held, table, steps
        # the memory of those that may move stays taken until they are seen to have moved: no other tensor gets its address
        self._watched, self._pinned = watched, [t.untyped_storage() for t in watched]
        self._places, self._indexes = [t.data_ptr() for t in watched], list(range(len(watched)))

    def _state(self, name, given, sizes, dtype, table, written):
        """A state's addresses in the table."""
        if given is None or len(given) != len(sizes):
            raise ValueError(f"{name} has one entry for each of params")
        device, each = self.device, dtype.itemsize
        for i, (t, k) in enumerate(zip(given, sizes)):
            if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != k:
                raise TypeError(f"{name}[{i}] must be a {dtype} CUDA tensor of {k} elements")
            at = _flat(t, name, i, device)
            setattr(table[i], name, at)
            written.append((at, k * each, name, i))

    def _take(self, grads, table, params):
        if len(grads) != len(params):
            raise ValueError("grads has one entry for each of params")
        device = self.device
        for i, (t, g, p) in enumerate(zip(table, grads, params)):
            t.grad_dtype = _code(g, "grads", i)
            if g.shape != p.shape:
                raise ValueError(f"grads[{i}] of shape {tuple(g.shape)} for a param of shape {tuple(p.shape)}")
            t.grad = _flat(g, "grads", i, device)

    def step(self, grads=None, *, lr=None, grad_scale=None, stream=None):
        """One step, of the gradients given or of those given at the start.

        lr: a number, or an fp32 CUDA tensor of one element (self.lr when None).
        grad_scale: an fp32 CUDA tensor of one element that every gradient is
        multiplied by (clipping), or None.  May be captured into a CUDA graph,
        of which each replay takes the next step.  The host's number for lr is
        then part of the graph; a tensor is read anew.
        """
        if lr is None:
            lr = self.lr
        if stream is not None:
            with torch.cuda.stream(stream):
                self.step(grads, lr=lr, grad_scale=grad_scale)
            held = self._held
            mine = [held["params"], held["master"], held["exp_avg"], held["exp_avg_sq"], held["exp_avg_scale"],
                    held["exp_avg_sq_scale"], held["grads"] if grads is None else grads,
                    [held["steps"], self._ticket, lr, grad_scale]]
            for t in (t for group in mine if group for t in group):
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
            return
        if torch.cuda.current_device() != self.device:
            raise ValueError(f"the optimizer is on cuda:{self.device}, but the current device is "
                             f"cuda:{torch.cuda.current_device()}")
        if not _unmoved(self._watched, self._places, self._indexes):
            self._lay()
        table, desc = self._table, self._desc
        if grads is not None:
            table = type(table)()
            ctypes.memmove(table, self._table, ctypes.sizeof(table))
            self._take(grads, table, self._held["params"])
        elif self._held["grads"] is None:
            raise ValueError("step needs the gradients: none were given at the start")
        if isinstance(lr, torch.Tensor):
            desc.lr, desc.lr_at = 0.0, _packed(lr, "lr", _F32, lr.shape if lr.numel() == 1 else (1,), self.device)
        else:
            desc.lr, desc.lr_at = lr, None
        desc.grad_scale = None if grad_scale is None else _packed(
            grad_scale, "grad_scale", _F32, grad_scale.shape if grad_scale.numel() == 1 else (1,), self.device)
        st = load_library().dgl_adamw(ctypes.byref(desc), table, len(table),
                                      torch._C._cuda_getCurrentRawStream(self.device))
        if st:
            _check(st, "dgl_adamw")
