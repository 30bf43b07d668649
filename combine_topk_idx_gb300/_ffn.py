"""Binding of the trained feed-forward block's products and of the clipping of
gradients.

Arguments are checked and marshalled here, nothing more.  A call with a layout's
handle has one matrix per expert; with ``handle=None`` there is one matrix and all
rows are in use (a shared expert).
"""
from __future__ import annotations

import bisect
import ctypes
import math
from typing import Optional, Sequence, Union

import torch

from ._binding import Handle
from ._ops import _BF16, _F32, _Call, _row_stride, _rows


def _matrix(c: _Call, handle: Optional[Handle], w: torch.Tensor, what: str, dtypes=_BF16):
    """(pointer, rows, columns) of a matrix, or of one per expert of the handle."""
    if w.dim() != (2 if handle is None else 3):
        raise ValueError(f"{what} must be " + ("a matrix" if handle is None
                                               else "one matrix per expert"))
    if handle is not None and w.shape[0] != handle.E:
        raise ValueError(f"{what} has {w.shape[0]} experts, the handle {handle.E}")
    return (c.ptr(w, what, dtypes), *w.shape[-2:])


def _strided(c: _Call, t: torch.Tensor, what: str, shape):
    """(pointer, row stride) of rows that may be strided."""
    return c.ptr(t, what, _BF16, shape, True), _row_stride(t, what)


def ep_ffn_gated(handle: Optional[Handle], x: torch.Tensor, w: torch.Tensor,
                 act: Optional[torch.Tensor] = None, gate_up: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """``silu(x Wg^T) * (x Wu^T)`` in one kernel (``ep_ffn_gated``): ``x`` BF16
    [rows, k] (may be row-strided), ``w`` BF16 [E, 2 * ffn, k] ([2 * ffn, k] without
    a handle), gate rows first.  Returns ``act`` BF16 [rows, ffn]; ``gate_up`` BF16
    [rows, 2 * ffn] is written if given, for :func:`ep_ffn_gated_backward`."""
    c = _Call("ep_ffn_gated", stream)
    hp, rows = _rows(handle, x, "x")
    wp, n, k = _matrix(c, handle, w, "w")
    if n % 2:
        raise ValueError(f"w has {n} rows, not gate and up alike")
    ffn = n // 2
    if act is None:
        act = c.empty(rows, ffn, dtype=torch.bfloat16)
    c(hp, rows, ffn, k, *_strided(c, x, "x", (rows, k)), wp, c.ptr(act, "act", _BF16, (rows, ffn)),
      c.ptr(gate_up, "gate_up", _BF16, (rows, n)))
    return act


def ep_ffn_gated_backward(handle: Optional[Handle], grad_out: torch.Tensor, w: torch.Tensor,
                          gate_up: torch.Tensor, grad_gate_up: Optional[torch.Tensor] = None,
                          act: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of ``gate_up`` through the down projection (``ep_ffn_gated_backward``):
    ``grad_out`` BF16 [rows, n] (may be row-strided), ``w`` BF16 [E, n, ffn] ([n, ffn]
    without a handle).  Returns ``grad_gate_up`` BF16 [rows, 2 * ffn]; ``act`` BF16
    [rows, ffn], the activation of gate and up as kept (rounded: not the forward's bits),
    is written if given."""
    c = _Call("ep_ffn_gated_backward", stream)
    hp, rows = _rows(handle, grad_out, "grad_out")
    wp, n, ffn = _matrix(c, handle, w, "w")
    if grad_gate_up is None:
        grad_gate_up = c.empty(rows, 2 * ffn, dtype=torch.bfloat16)
    c(hp, rows, ffn, n, *_strided(c, grad_out, "grad_out", (rows, n)), wp,
      c.ptr(gate_up, "gate_up", _BF16, (rows, 2 * ffn)),
      c.ptr(grad_gate_up, "grad_gate_up", _BF16, (rows, 2 * ffn)),
      c.ptr(act, "act", _BF16, (rows, ffn)))
    return grad_gate_up


def ep_ffn_product(handle: Optional[Handle], a: torch.Tensor, w: torch.Tensor,
                   out: Optional[torch.Tensor] = None, transposed: bool = False,
                   stream=None) -> torch.Tensor:
    """``a W^T`` with ``w`` BF16 [E, n, k], or with ``transposed`` ``a W`` with ``w``
    [E, k, n] (``ep_ffn_product``; no E without a handle): ``a`` BF16 [rows, k] (may
    be row-strided).  Returns BF16 [rows, n]."""
    c = _Call("ep_ffn_product", stream)
    hp, rows = _rows(handle, a, "a")
    wp, n, k = _matrix(c, handle, w, "w")
    if transposed:
        n, k = k, n
    if out is None:
        out = c.empty(rows, n, dtype=torch.bfloat16)
    c(hp, rows, n, k, *_strided(c, a, "a", (rows, k)), wp, int(bool(transposed)),
      c.ptr(out, "out", _BF16, (rows, n)))
    return out


def ep_ffn_weight_grad(handle: Optional[Handle], grad: torch.Tensor, a: torch.Tensor,
                       grad_w: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32,
                       accumulate: bool = False, stream=None) -> torch.Tensor:
    """Gradient of a projection's matrix (``ep_ffn_weight_grad``): the sum over each
    expert's rows (all rows without a handle) of ``grad[r]^T a[r]``, ``grad`` BF16
    [rows, n], ``a`` BF16 [rows, k] (both may be row-strided).  Returns ``grad_w``
    [E, n, k] ([n, k]), fp32 or BF16; a new one has ``dtype``.  With ``accumulate``
    the sum is added to the given ``grad_w``."""
    c = _Call("ep_ffn_weight_grad", stream)
    hp, rows = _rows(handle, grad, "grad")
    if a.dim() != 2:
        raise ValueError("a must have two dimensions")
    n, k = grad.shape[1], a.shape[1]
    if grad_w is None:
        if accumulate:
            raise ValueError("accumulate needs grad_w")
        if dtype not in _F32 + _BF16:
            raise ValueError(f"dtype {dtype}, expected {_F32 + _BF16}")
        lead = () if handle is None else (handle.E,)
        grad_w = c.empty(*lead, n, k, dtype=dtype)
    gp, gn, gk = _matrix(c, handle, grad_w, "grad_w", _F32 + _BF16)
    if (gn, gk) != (n, k):
        raise ValueError(f"grad_w shape {tuple(grad_w.shape)} does not end in {(n, k)}")
    c(hp, rows, n, k, *_strided(c, grad, "grad", (rows, n)), *_strided(c, a, "a", (rows, k)), gp,
      int(grad_w.dtype == torch.float32), int(bool(accumulate)))
    return grad_w


class _Memory:
    """The storages of tensors, each once, and where they were when they were listed.
    Holding a storage keeps its memory unless someone resizes it, which gives the memory
    back: :meth:`moved` says so."""

    def __init__(self, tensors):
        storages = (t.untyped_storage() for t in tensors)
        self.storages = list({s._cdata: s for s in storages}.values())
        self._at = list(map(torch.UntypedStorage.data_ptr, self.storages))
        self._bytes = list(map(torch.UntypedStorage.nbytes, self.storages))

    def moved(self) -> bool:
        # 0.12 us a storage; both, as one emptied and filled again may be where it was
        return (list(map(torch.UntypedStorage.data_ptr, self.storages)) != self._at
                or list(map(torch.UntypedStorage.nbytes, self.storages)) != self._bytes)

    def record_stream(self, stream):
        """The memory is in use on ``stream``."""
        for s in self.storages:
            torch.empty(0, dtype=torch.uint8, device=s.device).set_(s).record_stream(stream)


class GradPlan:
    """Gradients and where their clipped values go, listed once for many calls of
    :func:`ep_clip_grads`: a trainer's gradients stay where they are from step to
    step.  Holds the tensors and their storages, and reads nothing of them but on the
    GPU.  A tensor that is given another storage (``set_``, ``.data``) needs a new plan:
    this one goes on with the memory it listed.  A storage that is resized
    (``untyped_storage().resize_``, ``resize_`` to more than it holds) has given that
    memory back, and calls with the plan are refused.  With ``clips`` false it is for
    :func:`ep_grad_norm` only, and the gradients may overlap."""

    def __init__(self, grads: Sequence[torch.Tensor],
                 out: Optional[Sequence[torch.Tensor]] = None, clips: bool = True):
        self.clips = clips
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.out)} outputs for {len(self.grads)} gradients")
        self.device = None
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            for t, what in ((g, f"gradient {i}"), (o, f"output {i}")):
                if not t.is_cuda:
                    raise ValueError(f"{what} must be a CUDA tensor")
                if self.device is None:
                    self.device = t.get_device()
                if t.get_device() != self.device:
                    raise ValueError(f"{what} is on {t.device}, gradient 0 on cuda:{self.device}")
                if t.dtype not in _F32 + _BF16:
                    raise ValueError(f"{what} has dtype {t.dtype}, expected {_F32 + _BF16}")
                if not t.is_contiguous():
                    raise ValueError(f"{what} must be contiguous")
            if o.dtype != g.dtype or o.shape != g.shape:
                raise ValueError(f"output {i} is {o.dtype} {tuple(o.shape)}, its gradient "
                                 f"{g.dtype} {tuple(g.shape)}")
        n = len(self.grads)
        self._grads = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.grads])
        self._out = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.out])
        self._numels = (ctypes.c_int64 * n)(*[t.numel() for t in self.grads])
        self._f32 = (ctypes.c_uint8 * n)(*[t.dtype == torch.float32 for t in self.grads])
        # behind the addresses: data_ptr() gives a lazy copy memory of its own
        self._memory = _Memory(self.grads if out is None else self.grads + self.out)
        if clips:
            self._refuse_overlap()

    def _refuse_overlap(self):
        def spans(ts):
            return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i)
                    for i, t in enumerate(ts) if t.numel()]
        outs = sorted(spans(self.out))
        for a, b in zip(outs, outs[1:]):
            if b[0] < a[1]:
                raise ValueError(f"outputs {a[2]} and {b[2]} overlap")
        ends = [s[1] for s in outs]
        for lo, hi, i in spans(self.grads):
            k = bisect.bisect_right(ends, lo)  # the first output that ends behind lo
            while k < len(outs) and outs[k][0] < hi:
                if outs[k] != (lo, hi, i):
                    raise ValueError(f"gradient {i} overlaps output {outs[k][2]}")
                k += 1


def plan_grads(grads: Sequence[torch.Tensor],
               out: Optional[Sequence[torch.Tensor]] = None) -> GradPlan:
    """Lists ``grads`` (fp32 and BF16, contiguous) and where they are clipped to: in
    place, or into ``out``."""
    return GradPlan(grads, out)


def _clip(grads, max_norm, out, write, norm, stream):
    if isinstance(grads, GradPlan):
        if out is not None:
            raise ValueError("a plan has its outputs")
        plan = grads
        if plan._memory.moved():
            raise ValueError("a storage of the plan was resized: its tensors need a new plan")
        if write and not plan.clips:
            raise ValueError("the plan is for the norm only")
    else:
        plan = GradPlan(grads, out, write)
    max_norm = float(max_norm)
    if math.isnan(max_norm) or max_norm < 0:
        raise ValueError(f"max_norm = {max_norm}")
    c = _Call("ep_clip_grads", stream)
    if plan.device is not None and plan.device != c.device:
        raise ValueError(f"the gradients are on cuda:{plan.device}, the call runs on "
                         f"cuda:{c.device}")
    if c.other is not None:
        # the listed memory's, which the tensors may have left
        plan._memory.record_stream(c.other)
    if norm is None:
        norm = c.empty(dtype=torch.float32)
    c(len(plan.grads), plan._grads, plan._out if write else None, plan._numels, plan._f32,
      max_norm, c.ptr(norm, "norm", _F32, ()))
    return norm


def ep_grad_norm(grads: Union[GradPlan, Sequence[torch.Tensor]],
                 norm: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm of all gradients together, an fp32 tensor without dimensions on the
    GPU (``ep_clip_grads`` without outputs).  The same values may be in it twice."""
    return _clip(grads, math.inf, None, False, norm, stream)


def ep_clip_grads(grads: Union[GradPlan, Sequence[torch.Tensor]], max_norm: float,
                  out: Optional[Sequence[torch.Tensor]] = None,
                  norm: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scales all gradients by ``min(1, max_norm / (norm + 1e-6))``, in place or into
    ``out``, and returns their norm before that, an fp32 tensor without dimensions on
    the GPU (``ep_clip_grads``).  ``grads``: tensors, or a :func:`plan_grads` of them."""
    return _clip(grads, max_norm, out, True, norm, stream)
