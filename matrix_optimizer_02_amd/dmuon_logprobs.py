"""Python binding of the output head's log probabilities (include/dmuon_logprobs.h):
those of given tokens, with the entropy and the most likely alternatives of each
distribution, and their gradients, without keeping the logits of a large vocabulary.

    ws = workspace_for(tokens, hidden, vocab, torch.bfloat16, top_k=20)
    head_log_probs_forward(H, W, targets, logprobs, entropy, lse, top_ids, top_logprobs, workspace=ws)
    head_log_probs_backward(H, W, targets, lse, entropy, grad_logprobs, grad_entropy, grad_H, grad_W, workspace=ws)

top_ids and top_logprobs are what head_distill_forward takes as a teacher's entries,
grad_W what grad_norm_batched, grad_clip_batched and adamw_step_batched take.

The calls write into tensors that they are given and take no part in autograd:
inputs may require gradients, outputs carry no graph, and the gradients come from
the backward call alone.  Everything is computed by the library's HIP kernels.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .dmuon_head import HeadDesc, _grads, _problem, _tensor, _workspace
from .dmuon_ns import _DTYPE_CODE, _check, _lib, _stream_handle


def _declare():
    desc, vp, f32, i64, size = (ctypes.POINTER(HeadDesc), ctypes.c_void_p, ctypes.c_float, ctypes.c_int64,
                                ctypes.c_size_t)
    sig = {
        "head_log_probs_workspace_bytes": [desc, ctypes.c_int32, ctypes.POINTER(size)],
        "head_log_probs_forward": [desc, vp, vp, vp, i64, f32, vp, vp, vp, vp, vp, vp, size, vp],
        "head_log_probs_backward": [desc, vp, vp, vp, i64, f32, vp, vp, vp, vp, vp, vp, vp, size, vp],
    }
    for name, args in sig.items():
        fn = getattr(_lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args


_declare()


def workspace_bytes(tokens: int, hidden: int, vocab: int, dtype, *, top_k: int = 0, backward: bool = True) -> int:
    """Bytes of workspace for calls of at most ``tokens`` tokens: the forward
    call's with ``top_k`` alternatives, or with ``backward`` enough for both calls."""
    most = 0
    for b in (0, 1) if backward else (0,):
        d = HeadDesc(int(tokens), int(hidden), int(vocab), 0 if b else int(top_k), _DTYPE_CODE[dtype])
        n = ctypes.c_size_t()
        _check(_lib.head_log_probs_workspace_bytes(ctypes.byref(d), b, ctypes.byref(n)),
               "head_log_probs_workspace_bytes")
        most = max(most, n.value)
    return most


def workspace_for(tokens: int, hidden: int, vocab: int, dtype, *, top_k: int = 0, backward: bool = True,
                  device=None) -> torch.Tensor:
    """A device byte buffer of workspace_bytes (torch's allocator returns
    256-byte aligned blocks)."""
    n = workspace_bytes(tokens, hidden, vocab, dtype, top_k=top_k, backward=backward)
    return torch.empty(max(1, n), dtype=torch.uint8, device=device or "cuda")


def _maybe(t: Optional[torch.Tensor], what: str, shape, dtype):
    return None if t is None else _tensor(t, what, shape, dtype)


def head_log_probs_forward(hidden: torch.Tensor, weight: torch.Tensor, targets: Optional[torch.Tensor],
                           logprobs: Optional[torch.Tensor], entropy: Optional[torch.Tensor], lse: torch.Tensor,
                           top_ids: Optional[torch.Tensor] = None, top_logprobs: Optional[torch.Tensor] = None, *,
                           temperature: float = 1.0, ignore_index: int = -100, workspace: torch.Tensor = None,
                           stream=None) -> None:
    """Enqueue the log probabilities of ``targets`` (int64; None: of no token, and
    logprobs is None too), the entropies (None: not) and, with top_ids (tokens x K
    int64) and top_logprobs (tokens x K fp32), the K most likely alternatives.
    hidden (tokens x hidden) and weight (vocab x hidden) are bf16 or fp32;
    logprobs, entropy and lse (fp32, one a token) are written, 0 where the target
    is ignore_index (ids -1)."""
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    if (targets is None) != (logprobs is None):
        raise ValueError("targets and logprobs go together")
    if top_ids is not None and top_ids.dim() != 2:
        raise ValueError(f"top_ids: expected 2-D, got {tuple(top_ids.shape)}")
    k = 0 if top_ids is None else top_ids.shape[1]
    desc, (t, _, _), h, w = _problem(hidden, weight, k)
    f32, i64 = torch.float32, torch.int64
    args = (_maybe(targets, "targets", (t,), i64), int(ignore_index), float(temperature),
            _maybe(logprobs, "logprobs", (t,), f32), _maybe(entropy, "entropy", (t,), f32),
            _tensor(lse, "lse", (t,), f32), _maybe(top_ids if k else None, "top_ids", (t, k), i64),
            _maybe(top_logprobs if k else None, "top_logprobs", (t, k), f32), *_workspace(workspace))
    _check(_lib.head_log_probs_forward(ctypes.byref(desc), h, w, *args, _stream_handle(stream)),
           "head_log_probs_forward")


def head_log_probs_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: Optional[torch.Tensor],
                            lse: torch.Tensor, entropy: Optional[torch.Tensor], grad_logprobs: Optional[torch.Tensor],
                            grad_entropy: Optional[torch.Tensor], grad_hidden: Optional[torch.Tensor],
                            grad_weight: Optional[torch.Tensor], *, temperature: float = 1.0,
                            ignore_index: int = -100, workspace: torch.Tensor = None, stream=None) -> None:
    """Enqueue the gradients of sum(grad_logprobs logprobs) + sum(grad_entropy
    entropy): grad_hidden and grad_weight (of their matrix's dtype; either may be
    None) are overwritten.  lse and entropy are the forward call's; either of the
    upstream gradients may be None (entropy too where grad_entropy is)."""
    desc, shape, h, w = _problem(hidden, weight, 0)
    t, f32 = shape[0], torch.float32
    gh, gw = _grads(grad_hidden, grad_weight, shape, weight.dtype)
    args = (_maybe(targets, "targets", (t,), torch.int64), int(ignore_index), float(temperature),
            _tensor(lse, "lse", (t,), f32), _maybe(entropy, "entropy", (t,), f32),
            _maybe(grad_logprobs, "grad_logprobs", (t,), f32), _maybe(grad_entropy, "grad_entropy", (t,), f32), gh, gw,
            *_workspace(workspace))
    _check(_lib.head_log_probs_backward(ctypes.byref(desc), h, w, *args, _stream_handle(stream)),
           "head_log_probs_backward")


__all__ = ["workspace_bytes", "workspace_for", "head_log_probs_forward", "head_log_probs_backward"]
