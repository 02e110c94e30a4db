"""Python binding of the output-head losses (include/dmuon_head.h): softmax
cross entropy and distillation from a teacher's top logits over a large
vocabulary, forward and backward, without keeping the logits.

The entry points have the C ABI's names; this module turns torch tensors into
device pointers and the current torch stream into a hipStream_t.  Everything is
computed by the library's HIP kernels: there is no fallback.

    ws = workspace_for(tokens, hidden, vocab, torch.bfloat16)      # reused every step
    head_cross_entropy_forward(H, W, targets, losses, lse, workspace=ws)
    head_cross_entropy_backward(H, W, targets, lse, grad_losses, grad_H, grad_W, workspace=ws)

grad_W is what adamw_step_batched takes for the head.

The calls write into tensors that they are given and take no part in autograd:
inputs may require gradients, outputs carry no graph, and the gradients come from
the backward call alone.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .dmuon_ns import _DTYPE_CODE, _check, _lib, _on_current_device, _stream_handle


class HeadDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32)]


def _declare():
    desc, vp, f32, i64, size = (ctypes.POINTER(HeadDesc), ctypes.c_void_p, ctypes.c_float, ctypes.c_int64,
                                ctypes.c_size_t)
    sig = {
        "head_loss_workspace_bytes": [desc, ctypes.c_int32, ctypes.POINTER(size)],
        "head_cross_entropy_forward": [desc, vp, vp, vp, i64, vp, vp, vp, size, vp],
        "head_cross_entropy_backward": [desc, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, size, vp],
        "head_distill_forward": [desc, vp, vp, vp, vp, f32, vp, vp, vp, vp, size, vp],
        "head_distill_backward": [desc, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp, size, vp],
    }
    for name, args in sig.items():
        fn = getattr(_lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args


_declare()


def workspace_bytes(tokens: int, hidden: int, vocab: int, dtype, *, top_k: int = 0, backward: bool = True) -> int:
    """Bytes of workspace for calls of at most ``tokens`` tokens: the forward
    call's, or with ``backward`` enough for both calls."""
    d = HeadDesc(int(tokens), int(hidden), int(vocab), int(top_k), _DTYPE_CODE[dtype])
    most = 0
    for b in (0, 1) if backward else (0,):
        n = ctypes.c_size_t()
        _check(_lib.head_loss_workspace_bytes(ctypes.byref(d), b, ctypes.byref(n)), "head_loss_workspace_bytes")
        most = max(most, n.value)
    return most


def workspace_for(tokens: int, hidden: int, vocab: int, dtype, *, top_k: int = 0, backward: bool = True,
                  device=None) -> torch.Tensor:
    """A device byte buffer of workspace_bytes (torch's allocator returns
    256-byte aligned blocks)."""
    n = workspace_bytes(tokens, hidden, vocab, dtype, top_k=top_k, backward=backward)
    return torch.empty(max(1, n), dtype=torch.uint8, device=device or "cuda")


def _tensor(t: torch.Tensor, what: str, shape, dtype) -> ctypes.c_void_p:
    _on_current_device(t, what)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {'x'.join(map(str, shape))}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _problem(hidden: torch.Tensor, weight: torch.Tensor, top_k: int):
    """The descriptor of two matrices, and their pointers."""
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError(f"hidden {tuple(hidden.shape)} and weight {tuple(weight.shape)} must be 2-D with equal columns")
    if weight.dtype not in _DTYPE_CODE:
        raise ValueError("hidden and weight must be float32 or bfloat16")
    t, d, v = hidden.shape[0], hidden.shape[1], weight.shape[0]
    desc = HeadDesc(t, d, v, top_k, _DTYPE_CODE[weight.dtype])
    return desc, (t, d, v), _tensor(hidden, "hidden", (t, d), weight.dtype), _tensor(weight, "weight", (v, d),
                                                                                   weight.dtype)


def _workspace(ws: Optional[torch.Tensor]):
    if ws is None:
        raise ValueError("workspace is required (see workspace_for)")
    _on_current_device(ws, "workspace")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def _grads(grad_hidden, grad_weight, shape, dtype):
    t, d, v = shape
    gh = _tensor(grad_hidden, "grad_hidden", (t, d), dtype) if grad_hidden is not None else None
    gw = _tensor(grad_weight, "grad_weight", (v, d), dtype) if grad_weight is not None else None
    return gh, gw


def head_cross_entropy_forward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                               losses: torch.Tensor, lse: torch.Tensor, *, ignore_index: int = -100,
                               workspace: torch.Tensor = None, stream=None) -> None:
    """Enqueue the losses: hidden (tokens x hidden) and weight (vocab x hidden)
    bf16 or fp32, targets int64; losses and lse (fp32, one a token) are written,
    0 where the target is ignore_index."""
    desc, (t, _, _), h, w = _problem(hidden, weight, 0)
    f32 = torch.float32
    args = (_tensor(targets, "targets", (t,), torch.int64), int(ignore_index), _tensor(losses, "losses", (t,), f32),
            _tensor(lse, "lse", (t,), f32), *_workspace(workspace))
    _check(_lib.head_cross_entropy_forward(ctypes.byref(desc), h, w, *args, _stream_handle(stream)),
           "head_cross_entropy_forward")


def head_cross_entropy_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                                grad_losses: torch.Tensor, grad_hidden: Optional[torch.Tensor],
                                grad_weight: Optional[torch.Tensor], *, grad_lse: Optional[torch.Tensor] = None,
                                ignore_index: int = -100, workspace: torch.Tensor = None, stream=None) -> None:
    """Enqueue the gradients of sum(grad_losses losses) + sum(grad_lse lse):
    grad_hidden and grad_weight (of their matrix's dtype; either may be None) are
    overwritten.  lse is the forward call's."""
    desc, shape, h, w = _problem(hidden, weight, 0)
    t, f32 = shape[0], torch.float32
    gh, gw = _grads(grad_hidden, grad_weight, shape, weight.dtype)
    gl = _tensor(grad_lse, "grad_lse", (t,), f32) if grad_lse is not None else None
    args = (_tensor(targets, "targets", (t,), torch.int64), int(ignore_index), _tensor(lse, "lse", (t,), f32),
            _tensor(grad_losses, "grad_losses", (t,), f32), gl, gh, gw, *_workspace(workspace))
    _check(_lib.head_cross_entropy_backward(ctypes.byref(desc), h, w, *args, _stream_handle(stream)),
           "head_cross_entropy_backward")


def _teacher(teacher_ids, teacher_logits, t):
    if teacher_ids.dim() != 2:
        raise ValueError(f"teacher_ids: expected 2-D, got {tuple(teacher_ids.shape)}")
    k = teacher_ids.shape[1]
    return k, (_tensor(teacher_ids, "teacher_ids", (t, k), torch.int64),
               _tensor(teacher_logits, "teacher_logits", (t, k), torch.float32))


def head_distill_forward(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                         teacher_logits: torch.Tensor, losses: torch.Tensor, lse: torch.Tensor,
                         student_logits: torch.Tensor, *, temperature: float = 1.0,
                         workspace: torch.Tensor = None, stream=None) -> None:
    """Enqueue the distillation losses from teacher_ids (tokens x K int64,
    negative: absent) and teacher_logits (tokens x K fp32).  losses, lse and
    student_logits (tokens x K fp32) are written."""
    k, teacher = _teacher(teacher_ids, teacher_logits, hidden.shape[0])
    desc, (t, _, _), h, w = _problem(hidden, weight, k)
    f32 = torch.float32
    args = (*teacher, float(temperature), _tensor(losses, "losses", (t,), f32), _tensor(lse, "lse", (t,), f32),
            _tensor(student_logits, "student_logits", (t, k), f32), *_workspace(workspace))
    _check(_lib.head_distill_forward(ctypes.byref(desc), h, w, *args, _stream_handle(stream)), "head_distill_forward")


def head_distill_backward(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor,
                          teacher_logits: torch.Tensor, lse: torch.Tensor, student_logits: torch.Tensor,
                          grad_losses: torch.Tensor, grad_hidden: Optional[torch.Tensor],
                          grad_weight: Optional[torch.Tensor], *, temperature: float = 1.0,
                          workspace: torch.Tensor = None, stream=None) -> None:
    """Enqueue the gradients of sum(grad_losses losses); lse and student_logits
    are the forward call's, grad_hidden and grad_weight as for cross entropy."""
    k, teacher = _teacher(teacher_ids, teacher_logits, hidden.shape[0])
    desc, shape, h, w = _problem(hidden, weight, k)
    t, f32 = shape[0], torch.float32
    gh, gw = _grads(grad_hidden, grad_weight, shape, weight.dtype)
    args = (*teacher, float(temperature), _tensor(lse, "lse", (t,), f32),
            _tensor(student_logits, "student_logits", (t, k), f32), _tensor(grad_losses, "grad_losses", (t,), f32),
            gh, gw, *_workspace(workspace))
    _check(_lib.head_distill_backward(ctypes.byref(desc), h, w, *args, _stream_handle(stream)),
           "head_distill_backward")


__all__ = ["HeadDesc", "workspace_bytes", "workspace_for", "head_cross_entropy_forward",
           "head_cross_entropy_backward", "head_distill_forward", "head_distill_backward"]
