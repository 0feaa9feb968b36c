"""Binding of the AdamW step (include/bi_optim.h).  Argument checks and marshalling only."""
from __future__ import annotations

import ctypes
import operator
from typing import List, Optional, Sequence, Union

import numpy as np
import torch

from . import _lib
from .api import _ptr, _raise_host, _stream
from .attention import _on, _status

_nbytes, _shape, _dtype = (operator.attrgetter(a) for a in ("nbytes", "shape", "dtype"))
STATE_BLOCK = 256  # elements that share a scale in the 8-bit states


def _flat(ts, name, n, dtype, dev, sizes=None):
    if len(ts) != n:
        raise ValueError(f"{name} has {len(ts)} tensors, params has {n}")
    for i, t in enumerate(ts):
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"{name}[{i}] must be a CUDA tensor on {dev}, got {t.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name}[{i}] must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        if sizes is not None and t.numel() != sizes[i]:
            raise ValueError(f"{name}[{i}] must have {sizes[i]} elements, got {t.numel()}")


class AdamWState:
    """The tensors that ``adamw_step`` updates, checked once.

    ``params``: float32 or bfloat16, all of one type.  ``masters``: float32 weights of bfloat16 params
    (the update is made there and rounded into the param), or None.  ``exp_avg``, ``exp_avg_sq``:
    float32, or float8_e4m3fn with ``exp_avg_scale`` and ``exp_avg_sq_scale`` (float32, one for each
    256 elements): then m = exp_avg * scale and sqrt(v) = exp_avg_sq * scale.  A tensor that is replaced
    (``param.data = ...``) is checked anew at the next step: a param of another address, shape, type or layout,
    a state of another address or size in bytes."""

    def __init__(self, params: Sequence[torch.Tensor], masters: Optional[Sequence[torch.Tensor]],
                 exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor],
                 exp_avg_scale: Optional[Sequence[torch.Tensor]] = None,
                 exp_avg_sq_scale: Optional[Sequence[torch.Tensor]] = None):
        self._bind(params, masters, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale)

    def _bind(self, params, masters, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale):
        # into locals first: a handle that is bound again and refused stays what it was
        n = len(params)
        if n == 0:
            raise ValueError("params is empty")
        device = params[0].device
        if params[0].dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"params must be float32 or bfloat16, got {params[0].dtype}")
        param_bf16 = params[0].dtype == torch.bfloat16
        sizes = [p.numel() for p in params]
        _flat(params, "params", n, params[0].dtype, device)
        if masters is not None:
            if not param_bf16:
                raise ValueError("masters are for bfloat16 params")
            _flat(masters, "masters", n, torch.float32, device, sizes)
        if (exp_avg_scale is None) != (exp_avg_sq_scale is None):
            raise ValueError("exp_avg_scale and exp_avg_sq_scale are given together or not at all")
        state_bits = 32 if exp_avg_scale is None else 8
        held = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        _flat(exp_avg, "exp_avg", n, held, device, sizes)
        _flat(exp_avg_sq, "exp_avg_sq", n, held, device, sizes)
        if state_bits == 8:
            blocks = [-(-s // STATE_BLOCK) for s in sizes]
            _flat(exp_avg_scale, "exp_avg_scale", n, torch.float32, device, blocks)
            _flat(exp_avg_sq_scale, "exp_avg_sq_scale", n, torch.float32, device, blocks)
        lists = [None if ts is None else list(ts)
                 for ts in (params, masters, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale)]
        flat = [t for ts in lists if ts is not None for t in ts]
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in flat if t.numel())
        for (_, end), (start, _) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError("the tensors of one step may not overlap")
        # the rows of bi_adamw_tensor; the gradients' addresses are filled in at each step
        table = np.zeros((n, 8), dtype=np.int64)
        for i, ts in zip((0, 1, 3, 4, 5, 6), lists):
            if ts is not None:
                table[:, i] = [t.data_ptr() for t in ts]
        table[:, 7] = sizes
        self.device, self.param_bf16, self.state_bits = device, param_bf16, state_bits
        self.sizes, self.shapes = sizes, [p.shape for p in params]
        self.params, self.masters, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale = lists
        self._flat, self._ptrs, self._table = flat, [t.data_ptr() for t in flat], table
        # what the step writes, in order of addresses
        self._starts, self._ends = (np.array(x, dtype=np.int64) for x in (zip(*spans) if spans else ((0,), (0,))))
        self._grads = None  # addresses and element size that were held against them
        self._nbytes, self._dtypes = [t.nbytes for t in flat], [p.dtype for p in params]

    def _follow(self):
        """Tensors that are not what they were at the last step are checked again."""
        # All addresses and sizes in bytes, and what else a gradient is held to.  (57 parameters with masters and 32-bit
        # states: a step takes 69 us, with the addresses alone 44.  Types and layouts of the states would be more
        # still, and a state seen as another type or order of the same bytes is still the same memory.)
        params = self.params
        if (list(map(torch.Tensor.data_ptr, self._flat)) != self._ptrs or list(map(_nbytes, self._flat)) != self._nbytes or
                list(map(_shape, params)) != self.shapes or list(map(_dtype, params)) != self._dtypes or
                not all(map(torch.Tensor.is_contiguous, params))):
            self._bind(self.params, self.masters, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale,
                       self.exp_avg_sq_scale)

    def _rows(self, grads: Sequence[torch.Tensor], itemsize: int) -> np.ndarray:
        """The step's table."""
        ptrs = list(map(torch.Tensor.data_ptr, grads))
        self._table[:, 2] = ptrs
        if self._grads != (ptrs, itemsize):  # a matter of the addresses alone
            low, sizes = self._table[:, 2], self._table[:, 7]
            before = np.searchsorted(self._starts, low + sizes * itemsize) - 1  # the last that starts before the end
            if np.any((sizes > 0) & (before >= 0) & (self._ends[before] > low)):
                raise ValueError("a gradient may not overlap a tensor that the step writes")
            self._grads = ptrs, itemsize
        return self._table

    @staticmethod
    def allocate(params: Sequence[torch.Tensor], state_bits: int = 32, master: bool = False) -> "AdamWState":
        """States of zeros for ``params`` and, with ``master``, float32 copies of bfloat16 params."""
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        held = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        zeros = lambda: [torch.zeros(p.shape, dtype=torch.uint8 if state_bits == 8 else held,  # noqa: E731
                                     device=p.device).view(held) for p in params]
        scale = lambda: [torch.zeros(-(-p.numel() // STATE_BLOCK), device=p.device) for p in params]  # noqa: E731
        return AdamWState(params, [p.detach().float() for p in params] if master else None, zeros(), zeros(),
                          scale() if state_bits == 8 else None, scale() if state_bits == 8 else None)

    def tensors(self) -> List[torch.Tensor]:
        """Every tensor that a step reads and writes, the gradients apart."""
        lists = (self.params, self.masters, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)
        return [t for ts in lists if ts is not None for t in ts]


def adamw_step(state: AdamWState, grads: Sequence[torch.Tensor], step: Union[int, torch.Tensor], lr: float,
               beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """One AdamW step, in place, over all tensors of ``state`` (include/bi_optim.h).  ``grads``: one
    contiguous float32 or bfloat16 tensor (all of one type) for each param, of its shape.  ``step`` counts
    from 1; as a CUDA int64 tensor it is read when the kernel runs, so that a captured step can be
    replayed.  With 8-bit states, m of a beta1 above 17/18 and sqrt(v) of a beta2 above 0.96 (the default's, too)
    are rounded up or down by a fixed function of element and step, not to nearest: right on average, and
    scattered by about 20%.  ``grad_scale``: a CUDA float32 scalar that multiplies the gradients.  Returns status."""
    state._follow()  # before the gradients are held to the tensors' shapes
    dev = state.device
    n = len(state.params)
    if len(grads) != n:
        raise ValueError(f"grads has {len(grads)} tensors, params has {n}")
    gt = grads[0].dtype
    if gt not in (torch.float32, torch.bfloat16):
        raise ValueError(f"grads must be float32 or bfloat16, got {gt}")
    index = dev.index
    # whole lists at a time: with hundreds of small tensors the call is bound by these checks
    if ([g.shape for g in grads] != state.shapes or {g.dtype for g in grads} != {gt} or
            {g.get_device() for g in grads} != {index} or not all([g.is_contiguous() for g in grads])):
        for i, (g, shape) in enumerate(zip(grads, state.shapes)):
            if g.dtype is not gt or g.get_device() != index or g.shape != shape or not g.is_contiguous():
                raise ValueError(f"grads[{i}] must be a contiguous {gt} CUDA tensor of shape {list(shape)} on {dev}, got "
                                 f"{g.dtype} {list(g.shape)} on {g.device}")
    step_dev = None
    if isinstance(step, torch.Tensor):
        if not step.is_cuda or step.device != dev or step.dtype != torch.int64 or step.numel() != 1:
            raise ValueError(f"step must be an int or a CUDA int64 tensor of one element on {dev}")
        step_dev, step = step, 0
    if grad_scale is not None and (not grad_scale.is_cuda or grad_scale.device != dev or
                                   grad_scale.dtype != torch.float32 or grad_scale.numel() != 1):
        raise ValueError(f"grad_scale must be a CUDA float32 tensor of one element on {dev}")
    st = _status(status, dev)
    table = state._rows(grads, 4 if gt is torch.float32 else 2)
    cfg = _lib.AdamWCfg(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step),
                        state.state_bits, int(state.param_bf16), int(gt == torch.bfloat16), 0)
    with _on(dev):
        code = _lib.load().bi_adamw_step(table.ctypes.data, n, ctypes.addressof(cfg), _ptr(grad_scale),
                                         _ptr(step_dev), _ptr(st), _stream(dev))
    _raise_host(code, "bi_adamw_step")
    return st
