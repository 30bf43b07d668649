"""Binding of the operators around dispatch and combine: the norm before the
dispatch, the experts' products and the gated activation between them, and the
gradient of the weighted combine.

Like the rest of the binding this only checks and marshals arguments.  Every
call is ordered on the current torch stream, or on ``stream=``; a tensor that
belongs to another stream is recorded on that one, so its memory is not reused
while the call still runs.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import EP_OK, EpError, Handle, load_library

_FP8 = (torch.uint8, torch.float8_e4m3fn)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)


class _Call:
    """One call's stream, device check and tensor pointers."""

    __slots__ = ("fn", "name", "raw", "other", "device")

    def __init__(self, name: str, stream):
        self.name = name
        self.fn = getattr(load_library(), name)
        self.device = torch.cuda.current_device()
        # the raw handle: making a torch Stream of the current one takes 2.8 us, most of a launch
        current = torch._C._cuda_getCurrentRawStream(self.device)
        self.other = None
        if stream is None:
            self.raw = current
        else:
            self.raw = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
            if self.raw != current:
                # the default stream's handle is 0, of which ExternalStream makes a new stream
                self.other = (torch.cuda.ExternalStream(self.raw) if self.raw
                              else torch.cuda.default_stream(self.device))

    def ptr(self, t: Optional[torch.Tensor], what: str, dtypes: tuple, shape=None, strided=False):
        """Pointer of an optional tensor of the expected type and shape."""
        if t is None:
            return None
        if (t.get_device() != self.device or t.dtype not in dtypes
                or (shape is not None and t.shape != shape)
                or not (strided or t.is_contiguous())):
            self.refuse(t, what, dtypes, shape)
        if self.other is not None:
            t.record_stream(self.other)
        return t.data_ptr() or None

    def refuse(self, t, what, dtypes, shape):
        if not t.is_cuda:
            raise ValueError(f"{what} must be a CUDA tensor")
        if t.get_device() != self.device:
            raise ValueError(f"{what} is on {t.device}, the call runs on cuda:{self.device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{what} has dtype {t.dtype}, expected {dtypes}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{what} shape {tuple(t.shape)} != {tuple(shape)}")
        raise ValueError(f"{what} must be contiguous")

    def empty(self, *shape, dtype):
        """An output tensor of the call's stream."""
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device="cuda")
        with torch.cuda.stream(self.other):
            return torch.empty(shape, dtype=dtype, device="cuda")

    def __call__(self, *args):
        st = self.fn(*args, self.raw)
        if st != EP_OK:
            raise EpError(st, self.name)


def sf_layout(handle: Handle, n: int):
    """(numel, token_stride, hidden_stride, expert_stride) of the fp32 scales of
    rows of ``n`` elements in the handle's layout (``ep_sf_layout``)."""
    ptr = handle.ptr
    known = handle.sf_layouts.get(n)  # fixed for the handle's life
    if known is None:
        v = [ctypes.c_int64() for _ in range(4)]
        st = load_library().ep_sf_layout(ptr, n, *map(ctypes.byref, v))
        if st != EP_OK:
            raise EpError(st, "ep_sf_layout")
        known = handle.sf_layouts[n] = tuple(x.value for x in v)
    return known


def alloc_fp8(handle: Handle, n: int, zero: bool = False):
    """(e4m3 bytes [rows_alloc, n], flat fp32 scales) in the handle's layout."""
    mk = torch.zeros if zero else torch.empty
    return (mk((handle.rows_alloc, n), dtype=torch.uint8, device="cuda"),
            mk((sf_layout(handle, n)[0],), dtype=torch.float32, device="cuda"))


def alloc_rmsnorm(x: torch.Tensor, residual: bool = False, bf16: bool = False, fp8: bool = True,
                  col_major_sf: bool = False, rstd: bool = False) -> dict:
    """Outputs of :func:`ep_rmsnorm` for ``x`` [T, H].  The scales are a [T, H / 128]
    view, column-major with 16-byte aligned columns if ``col_major_sf``: both
    forms are what :func:`ep_dispatch_fp8` takes."""
    T, H = x.shape
    # of x's shape by empty_like: half the time of torch.empty, and a small call is mostly this
    like, dense, f32 = torch.empty_like, torch.contiguous_format, torch.float32
    out = {"residual_out": like(x, memory_format=dense) if residual else None,
           "y": like(x, memory_format=dense) if bf16 else None, "y_fp8": None, "y_sf": None,
           "rstd": x.new_empty((T,), dtype=f32) if rstd else None}
    if fp8:
        out["y_fp8"] = like(x, dtype=torch.uint8, memory_format=dense)
        if col_major_sf:
            # not a view of a larger tensor: slicing and transposing one takes 6 us more
            out["y_sf"] = x.new_empty_strided((T, H // 128), (1, max(4, -(-T // 4) * 4)), dtype=f32)
        else:
            out["y_sf"] = x.new_empty((T, H // 128), dtype=f32)
    return out


def _row_stride(t: torch.Tensor, what: str) -> int:
    T, H = t.shape
    row, col = t.stride()
    if col != 1 and H > 1 and T > 0:
        raise ValueError(f"{what} must be dense within a row")
    return row if T > 1 and H > 0 else -(-H // 8) * 8


def _gamma(c: _Call, gamma: torch.Tensor, H: int):
    return c.ptr(gamma, "gamma", _BF16 + _F32, (H,)), int(gamma.dtype == torch.float32)


def ep_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float,
               residual: Optional[torch.Tensor] = None,
               residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               y_fp8: Optional[torch.Tensor] = None, y_sf: Optional[torch.Tensor] = None,
               rstd: Optional[torch.Tensor] = None, stream=None) -> None:
    """Root-mean-square norm of ``x + residual`` into the given outputs (``ep_rmsnorm``).

    ``x`` and ``residual`` are BF16 [T, H] and may be row-strided; ``gamma`` is
    BF16 or fp32 [H].  ``residual_out`` may be ``residual`` itself."""
    c = _Call("ep_rmsnorm", stream)
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    shape = x.shape
    xp = c.ptr(x, "x", _BF16, None, True)
    rp = c.ptr(residual, "residual", _BF16, shape, True)
    gp, f32 = _gamma(c, gamma, H)
    ts = hs = 0
    sp = None
    if y_sf is not None:
        sp = c.ptr(y_sf, "y_sf", _F32, (T, H // 128), True)
        ts, hs = y_sf.stride()
        if (ts == 0 and T > 1) or (hs == 0 and H >= 256):
            raise ValueError("y_sf must not be an expanded tensor")
        ts, hs = ts or 1, hs or 1
    c(T, H, xp, _row_stride(x, "x"), rp,
      0 if residual is None else _row_stride(residual, "residual"), gp, f32, eps,
      c.ptr(residual_out, "residual_out", _BF16, shape), c.ptr(y, "y", _BF16, shape),
      c.ptr(y_fp8, "y_fp8", _FP8, shape), sp, ts, hs, c.ptr(rstd, "rstd", _F32, (T,)))


def ep_rmsnorm_backward(grad_y: torch.Tensor, normed: torch.Tensor, gamma: torch.Tensor,
                        rstd: torch.Tensor, grad_residual: Optional[torch.Tensor] = None,
                        grad_x: Optional[torch.Tensor] = None,
                        grad_gamma: Optional[torch.Tensor] = None, need_gamma: bool = True,
                        stream=None):
    """Gradient of :func:`ep_rmsnorm`; ``normed`` is its ``residual_out`` (or ``x``
    without a residual).  Returns (grad_x BF16 [T, H], grad_gamma fp32 [H] or
    None without ``need_gamma``)."""
    c = _Call("ep_rmsnorm_backward", stream)
    if normed.dim() != 2:
        raise ValueError("normed must be [T, H]")
    T, H = normed.shape
    if grad_x is None:
        grad_x = c.empty(T, H, dtype=torch.bfloat16)
    if grad_gamma is None and need_gamma:
        grad_gamma = c.empty(H, dtype=torch.float32)
    gp, f32 = _gamma(c, gamma, H)
    c(T, H, c.ptr(grad_y, "grad_y", _BF16, normed.shape), c.ptr(normed, "normed", _BF16), gp, f32,
      c.ptr(rstd, "rstd", _F32, (T,)),
      c.ptr(grad_residual, "grad_residual", _BF16, normed.shape),
      c.ptr(grad_x, "grad_x", _BF16, normed.shape), c.ptr(grad_gamma, "grad_gamma", _F32, (H,)))
    return grad_x, grad_gamma


def _rows(handle: Optional[Handle], t: torch.Tensor, what: str):
    """(handle pointer, rows) of a call on a layout's rows, or on all rows of ``t``."""
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    if handle is None:
        return None, t.shape[0]
    return handle.ptr, handle.rows_alloc


def _sf_numel(handle: Optional[Handle], rows: int, n: int):
    return (rows, n // 128) if handle is None else (sf_layout(handle, n)[0],)


def ep_swiglu(handle: Optional[Handle], gate_up: torch.Tensor,
              row_weights: Optional[torch.Tensor] = None, act: Optional[torch.Tensor] = None,
              act_fp8: Optional[torch.Tensor] = None, act_sf: Optional[torch.Tensor] = None,
              ckpt: Optional[torch.Tensor] = None, ckpt_sf: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """Gated activation of the handle's rows (all rows without a handle) into the
    given outputs (``ep_swiglu``): ``act`` BF16, ``act_fp8`` with flat scales
    ``act_sf`` in the handle's layout ([rows, ffn / 128] without one), and the
    8-bit checkpoint ``ckpt`` [rows, 2 * ffn] with ``ckpt_sf`` [rows, 2 * ffn / 128]."""
    c = _Call("ep_swiglu", stream)
    hp, rows = _rows(handle, gate_up, "gate_up")
    F = gate_up.shape[1] // 2
    gp = c.ptr(gate_up, "gate_up", _BF16, (rows, 2 * F))
    c(hp, rows, F, gp, c.ptr(row_weights, "row_weights", _F32, (rows,)),
      c.ptr(act, "act", _BF16, (rows, F)), c.ptr(act_fp8, "act_fp8", _FP8, (rows, F)),
      None if act_sf is None else c.ptr(act_sf, "act_sf", _F32, _sf_numel(handle, rows, F)),
      c.ptr(ckpt, "ckpt", _FP8, (rows, 2 * F)),
      c.ptr(ckpt_sf, "ckpt_sf", _F32, (rows, 2 * F // 128)))


def ep_swiglu_backward(handle: Optional[Handle], grad_act: torch.Tensor, ckpt: torch.Tensor,
                       ckpt_sf: torch.Tensor, row_weights: Optional[torch.Tensor] = None,
                       grad_gate_up: Optional[torch.Tensor] = None,
                       grad_fp8: Optional[torch.Tensor] = None,
                       grad_sf: Optional[torch.Tensor] = None,
                       grad_row_weights: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradient of :func:`ep_swiglu` from its checkpoint into the given outputs
    (``ep_swiglu_backward``)."""
    c = _Call("ep_swiglu_backward", stream)
    hp, rows = _rows(handle, grad_act, "grad_act")
    F = grad_act.shape[1]
    c(hp, rows, F, c.ptr(grad_act, "grad_act", _BF16, (rows, F)),
      c.ptr(ckpt, "ckpt", _FP8, (rows, 2 * F)),
      c.ptr(ckpt_sf, "ckpt_sf", _F32, (rows, 2 * F // 128)),
      c.ptr(row_weights, "row_weights", _F32, (rows,)),
      c.ptr(grad_gate_up, "grad_gate_up", _BF16, (rows, 2 * F)),
      c.ptr(grad_fp8, "grad_fp8", _FP8, (rows, 2 * F)),
      None if grad_sf is None else c.ptr(grad_sf, "grad_sf", _F32,
                                         _sf_numel(handle, rows, 2 * F)),
      c.ptr(grad_row_weights, "grad_row_weights", _F32, (rows,)))


def ep_combine_weighted_backward(handle: Handle, grad_out: torch.Tensor,
                                 y: Optional[torch.Tensor], topk_weights: torch.Tensor,
                                 expert_bias: Optional[torch.Tensor] = None,
                                 grad_y: Optional[torch.Tensor] = None,
                                 grad_y_fp8: Optional[torch.Tensor] = None,
                                 grad_y_sf: Optional[torch.Tensor] = None,
                                 grad_topk_weights: Optional[torch.Tensor] = None,
                                 grad_expert_bias: Optional[torch.Tensor] = None,
                                 stream=None) -> None:
    """Gradient of :func:`ep_combine` with weights into the given outputs
    (``ep_combine_weighted_backward``)."""
    c = _Call("ep_combine_weighted_backward", stream)
    T, K, E, H, rows = handle.T, handle.K, handle.E, handle.H, handle.rows_alloc
    c(handle.ptr, c.ptr(grad_out, "grad_out", _BF16, (T, H)),
      c.ptr(y, "y", _BF16, (rows, H)), c.ptr(topk_weights, "topk_weights", _F32, (T, K)),
      c.ptr(expert_bias, "expert_bias", _BF16, (E, H)), c.ptr(grad_y, "grad_y", _BF16, (rows, H)),
      c.ptr(grad_y_fp8, "grad_y_fp8", _FP8, (rows, H)),
      None if grad_y_sf is None else c.ptr(grad_y_sf, "grad_y_sf", _F32,
                                           (sf_layout(handle, H)[0],)),
      c.ptr(grad_topk_weights, "grad_topk_weights", _F32, (T, K)),
      c.ptr(grad_expert_bias, "grad_expert_bias", _F32, (E, H)))


def ep_expert_gemm(handle: Handle, a: torch.Tensor, a_sf: torch.Tensor, w: torch.Tensor,
                   w_sf: torch.Tensor, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The experts' FP8 product over the handle's expanded rows (``ep_expert_gemm``):
    ``a`` e4m3 [rows_alloc, k] with flat scales in the handle's layout, ``w`` e4m3
    [E, n, k] with ``w_sf`` fp32 [E, ceil(n / 128), k / 128]; returns BF16
    [rows_alloc, n]."""
    c = _Call("ep_expert_gemm", stream)
    if w.dim() != 3:
        raise ValueError("w must be [E, n, k]")
    E, n, k = w.shape
    if E != handle.E:
        raise ValueError(f"w has {E} experts, the handle {handle.E}")
    if k % 128 or k == 0:
        raise ValueError(f"k = {k} is not a multiple of 128")
    rows = handle.rows_alloc
    if out is None:
        out = c.empty(rows, n, dtype=torch.bfloat16)
    c(handle.ptr, n, k, c.ptr(a, "a", _FP8, (rows, k)),
      c.ptr(a_sf, "a_sf", _F32, (sf_layout(handle, k)[0],)), c.ptr(w, "w", _FP8),
      c.ptr(w_sf, "w_sf", _F32, (E, -(-n // 128), k // 128)),
      c.ptr(out, "out", _BF16, (rows, n)))
    return out
