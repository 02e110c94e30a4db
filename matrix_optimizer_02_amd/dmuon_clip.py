"""Python binding of the gradient norm and clipping (include/dmuon_clip.h).

    norm = torch.empty((), device="cuda")
    grad_norm_batched(grads, norm, workspace=norm_workspace_for(grads))
    grad_clip_batched(grads, norm, 1.0)                  # in place; then the optimizer's step

or, for gradients that stay where they are from step to step (zeroed in place: their
sizes, types and addresses are gathered once):

    batch = GradBatch(grads)
    batch.norm(norm)
    batch.clip(norm, 1.0)

Owners of different tensors join their norms between the two calls: the norm of
all is the root of the sum of their squares.  Everything is computed by the
library's HIP kernels, nothing waits for the device, and the calls take no part in
autograd.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from .dmuon_ns import _DTYPE_CODE, _check, _lib, _on_current_device, _stream_handle


def _declare():
    i32, vp, vpp, f64 = ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p), ctypes.c_double
    i64p, i32p, size = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32), ctypes.c_size_t
    sig = {
        "grad_norm_workspace_bytes": [i32, i64p, i32p, ctypes.POINTER(size)],
        "grad_norm_batched": [i32, i64p, i32p, vpp, vp, vp, size, vp],
        "grad_clip_batched": [i32, i64p, i32p, vpp, vpp, vp, f64, f64, vp],
    }
    for name, args in sig.items():
        fn = getattr(_lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args


_declare()


_address = torch.Tensor.data_ptr


class _Table:
    """The host arrays of a list of tensors: sizes, types and addresses."""

    def __init__(self, tensors: Sequence[torch.Tensor], what: str):
        for i, t in enumerate(tensors):
            _on_current_device(t, f"{what}[{i}]")
            if not t.is_contiguous():
                raise ValueError(f"{what}[{i}] must be contiguous")
            if t.dtype not in _DTYPE_CODE:
                raise ValueError(f"{what}[{i}]: must be float32 or bfloat16, got {t.dtype}")
        n = self.count = len(tensors)
        self.device = tensors[0].device if n else None
        self.numels = (ctypes.c_int64 * max(1, n))(*[t.numel() for t in tensors])
        self.dtypes = (ctypes.c_int32 * max(1, n))(*[_DTYPE_CODE[t.dtype] for t in tensors])
        self.addresses = list(map(_address, tensors))
        self.pointers = (ctypes.c_void_p * max(1, n))(*self.addresses)

    def check(self, tensors: Sequence[torch.Tensor], what: str) -> None:
        """The tensors still lie where they were, on the device that is current."""
        if self.device is not None and self.device.index != torch.cuda.current_device():
            raise ValueError(f"{what} are on {self.device}; the current device is cuda:{torch.cuda.current_device()}")
        if list(map(_address, tensors)) != self.addresses:
            i = next(i for i, (t, a) in enumerate(zip(tensors, self.addresses)) if t.data_ptr() != a)
            raise ValueError(f"{what}[{i}] does not lie where it was when the batch was built; build another one")


def _outputs(grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]], table: _Table) -> _Table:
    if outs is None:
        return table
    if len(outs) != len(grads):
        raise ValueError(f"outs: expected {len(grads)} tensors, got {len(outs)}")
    for i, (g, o) in enumerate(zip(grads, outs)):
        if o.shape != g.shape or o.dtype is not g.dtype:
            raise ValueError(f"outs[{i}]: expected {g.dtype} {tuple(g.shape)}, got {o.dtype} {tuple(o.shape)}")
    return _Table(outs, "outs")


def _here(t: torch.Tensor, what: str) -> None:
    # (the short way of what follows, for calls of a few microseconds)
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        _on_current_device(t, what)


def _scalar(norm: torch.Tensor) -> ctypes.c_void_p:
    _here(norm, "norm")
    if norm.numel() != 1 or norm.dtype is not torch.float32:
        raise ValueError(f"norm: expected one float32, got {norm.dtype} {tuple(norm.shape)}")
    return ctypes.c_void_p(norm.data_ptr())


def _workspace_bytes(table: _Table) -> int:
    n = ctypes.c_size_t()
    _check(_lib.grad_norm_workspace_bytes(table.count, table.numels, table.dtypes, ctypes.byref(n)),
           "grad_norm_workspace_bytes")
    return n.value


def _norm(table: _Table, norm, workspace, stream):
    if workspace is None:
        raise ValueError("workspace is required (see norm_workspace_for)")
    _here(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check(_lib.grad_norm_batched(table.count, table.numels, table.dtypes, table.pointers, _scalar(norm),
                                  ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream)), "grad_norm_batched")


def _clip(table: _Table, outs: _Table, norm, max_norm, eps, stream):
    _check(_lib.grad_clip_batched(table.count, table.numels, table.dtypes, table.pointers, outs.pointers,
                                  _scalar(norm), float(max_norm), float(eps), _stream_handle(stream)),
           "grad_clip_batched")


def norm_workspace_for(grads: Sequence[torch.Tensor], device=None) -> torch.Tensor:
    """A device byte buffer for grad_norm_batched over tensors of these sizes and
    types, wherever they begin (torch's allocator returns 256-byte aligned blocks)."""
    return torch.empty(max(1, _workspace_bytes(_Table(grads, "grads"))), dtype=torch.uint8, device=device or "cuda")


def grad_norm_batched(grads: Sequence[torch.Tensor], norm: torch.Tensor, *, workspace: torch.Tensor = None,
                      stream=None) -> None:
    """Enqueue the global 2-norm of a list of bf16 and fp32 tensors (contiguous,
    beginning at any element) into ``norm``, one fp32 on the device."""
    _norm(_Table(grads, "grads"), norm, workspace, stream)


def grad_clip_batched(grads: Sequence[torch.Tensor], norm: torch.Tensor, max_norm: float,
                      outs: Optional[Sequence[torch.Tensor]] = None, *, eps: float = 1e-6, stream=None) -> None:
    """Enqueue g min(1, max_norm / (norm + eps)) for every tensor, in place or into
    ``outs`` (of the same shapes and types)."""
    table = _Table(grads, "grads")
    _clip(table, _outputs(grads, outs, table), norm, max_norm, eps, stream)


class GradBatch:
    """A list of gradients that stay where they are (and, to clip into other buffers,
    their outputs), with the norm's workspace.  The batch keeps the tensors alive;
    its calls on different streams must not overlap in time.

    Every call is refused where a tensor's memory was replaced since (``.data``,
    ``set_``, a resized storage) or another device is current.  A parameter that was
    given a new ``.grad`` tensor is not seen: zero gradients in place
    (``zero_grad(set_to_none=False)``), or take the list calls."""

    def __init__(self, grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None):
        self._grads, self._outs = list(grads), None if outs is None else list(outs)
        self._table = _Table(self._grads, "grads")
        self._to = _outputs(self._grads, self._outs, self._table)
        self.workspace = torch.empty(max(1, _workspace_bytes(self._table)), dtype=torch.uint8,
                                     device=self._table.device or "cuda")

    def norm(self, norm: torch.Tensor, *, stream=None) -> None:
        self._table.check(self._grads, "grads")
        _norm(self._table, norm, self.workspace, stream)

    def clip(self, norm: torch.Tensor, max_norm: float, *, eps: float = 1e-6, stream=None) -> None:
        self._table.check(self._grads, "grads")
        if self._outs is not None:
            self._to.check(self._outs, "outs")
        _clip(self._table, self._to, norm, max_norm, eps, stream)


__all__ = ["norm_workspace_for", "grad_norm_batched", "grad_clip_batched", "GradBatch"]
