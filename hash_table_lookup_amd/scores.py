"""Losses of a softmax over a whole vocabulary, which never hold the scores of all rows with all items.

A row is scored against every row of a vocabulary (the items that can follow
it): s[i, v] = x[i] @ w[v] / temperature.  :func:`softmax_loss` is the cross
entropy with one item each, :func:`distill_loss` the divergence from a
teacher's top logits.  Gradients are functions of their own, as the library's
backward calls are; a row without a target (an index outside the vocabulary)
has loss and gradients of zero, whatever it holds.
"""
from __future__ import annotations

from typing import Tuple

import torch

from ._binding import _TORCH_DTYPE, _check, _dev, _dtype_code, _ptr, _stream, lib
from .dense import _here, _rows, _scratch

_VOCAB_MAX = 1 << 30
_TOP_MAX = 1024


def _pair(x: torch.Tensor, w: torch.Tensor):
    """(x, its row stride, w, its row stride) of one type and row length."""
    x, ldx = _rows(x, "x")
    w, ldw = _rows(w, "w", dtype=x.dtype)
    if w.shape[1] != x.shape[1]:
        raise ValueError(f"x has rows of {x.shape[1]}, w of {w.shape[1]}")
    if not 1 <= w.shape[0] <= _VOCAB_MAX:
        raise ValueError(f"w must have 1 to {_VOCAB_MAX} rows, got {w.shape[0]}")
    return x, ldx, w, ldw


def _indices(t: torch.Tensor, shape, name: str) -> Tuple[torch.Tensor, int]:
    if not t.is_cuda or t.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"{name} must be a GPU tensor of int32 or int64, got {t.dtype} on {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.contiguous(), 32 if t.dtype == torch.int32 else 64


def _floats(t: torch.Tensor, shape, name: str) -> torch.Tensor:
    t = _dev(t, torch.float32, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _heat(temperature: float) -> float:
    temperature = float(temperature)
    if not 1e-30 <= temperature <= 1e30:
        raise ValueError(f"temperature must be in [1e-30, 1e30], got {temperature}")
    return temperature


def softmax_loss(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, temperature: float = 1.0):
    """Cross entropy of each row against a vocabulary (softmax_loss).

    x [m, k], w [vocab, k] of one type, targets [m] int32 or int64.  Returns
    (loss, lse), both float32 [m]: lse[i] = log sum_v exp(s[i, v]), which
    softmax_loss_backward takes, and loss[i] = lse[i] - s[i, targets[i]]; both
    are 0 for a row whose target is outside the vocabulary."""
    heat = _heat(temperature)
    x, ldx, w, ldw = _pair(x, w)
    m, k = x.shape
    targets, bits = _indices(targets, (m,), "targets")
    _here(x, w, targets)
    loss, lse = (torch.empty(m, dtype=torch.float32, device=x.device) for _ in range(2))
    nb = lib().softmax_loss_workspace_bytes(m, w.shape[0], k, _dtype_code(x.dtype))
    ws = _scratch("softmax_loss", nb, x.device)
    _check(lib().softmax_loss(_ptr(x), ldx, _ptr(w), ldw, _dtype_code(x.dtype), m, w.shape[0], k, _ptr(targets), bits,
                              heat, _ptr(loss), _ptr(lse), _ptr(ws), nb, _stream()))
    return loss, lse


def softmax_loss_backward(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                          lse: torch.Tensor, temperature: float = 1.0, dx_dtype=None, need_dx: bool = True,
                          need_dw: bool = True):
    """(dx [m, k] in ``dx_dtype`` (x's), dw [vocab, k] in w's type) of softmax_loss; None for one not needed.

    dloss float32 [m] is the gradient of each row's loss, lse what
    softmax_loss returned at the same x, w and temperature."""
    heat = _heat(temperature)
    x, ldx, w, ldw = _pair(x, w)
    (m, k), vocab, d = x.shape, w.shape[0], x.device
    targets, bits = _indices(targets, (m,), "targets")
    dloss, lse = _floats(dloss, (m,), "dloss"), _floats(lse, (m,), "lse")
    _here(x, w, targets, dloss, lse)
    code, dtype = _dtype_code(x.dtype if dx_dtype is None else dx_dtype), _dtype_code(x.dtype)
    dx = torch.empty((m, k), dtype=_TORCH_DTYPE[code], device=d) if need_dx else None
    dw = torch.empty((vocab, k), dtype=x.dtype, device=d) if need_dw else None
    nb = lib().softmax_loss_backward_workspace_bytes(m, vocab, k, dtype)
    ws = _scratch("softmax_loss_backward", nb, d)
    _check(lib().softmax_loss_backward(_ptr(dloss), _ptr(x), ldx, _ptr(w), ldw, dtype, m, vocab, k, _ptr(targets), bits,
                                       _ptr(lse), heat, _ptr(dx), code, _ptr(dw), _ptr(ws), nb, _stream()))
    return dx, dw


def _lists(top: torch.Tensor, top_logits: torch.Tensor, m: int):
    """(items, index bits, logits, their row stride, list length) of a teacher."""
    if top.dim() != 2 or not 1 <= top.shape[1] <= _TOP_MAX:
        raise ValueError(f"top must have shape [{m}, 1 to {_TOP_MAX}], got {tuple(top.shape)}")
    items, bits = _indices(top, (m, top.shape[1]), "top")
    logits, ld = _rows(top_logits, "top_logits")
    if tuple(logits.shape) != tuple(items.shape):
        raise ValueError(f"top_logits must have shape {tuple(items.shape)}, got {tuple(logits.shape)}")
    return items, bits, logits, ld, items.shape[1]


def distill_loss(x: torch.Tensor, w: torch.Tensor, top: torch.Tensor, top_logits: torch.Tensor,
                 temperature: float = 1.0):
    """Divergence of each row's softmax over a vocabulary from a teacher's top logits (distill_loss).

    top [m, t] (int32 or int64) lists a teacher's items of each row, top_logits
    [m, t] (float32 or bfloat16) its logits; an index outside the vocabulary
    is no entry.  With p the softmax of a row's listed logits / temperature,
    loss[i] = sum_j p[j] (log p[j] - log q[top[i, j]]), q the row's softmax.
    Returns (loss float32 [m], kept): kept, which distill_loss_backward takes,
    is (lse [m], the scores [m, t] of the listed items).  Scale by
    temperature**2 where the gradient's size should not depend on it."""
    heat = _heat(temperature)
    x, ldx, w, ldw = _pair(x, w)
    m, k = x.shape
    items, bits, logits, ld, t = _lists(top, top_logits, m)
    _here(x, w, items, logits)
    loss, lse = (torch.empty(m, dtype=torch.float32, device=x.device) for _ in range(2))
    scores = torch.empty((m, t), dtype=torch.float32, device=x.device)
    nb = lib().softmax_loss_workspace_bytes(m, w.shape[0], k, _dtype_code(x.dtype))
    ws = _scratch("softmax_loss", nb, x.device)
    _check(lib().distill_loss(_ptr(x), ldx, _ptr(w), ldw, _dtype_code(x.dtype), m, w.shape[0], k, _ptr(items), bits,
                              _ptr(logits), _dtype_code(logits.dtype), ld, t, heat, _ptr(loss), _ptr(lse), _ptr(scores),
                              _ptr(ws), nb, _stream()))
    return loss, (lse, scores)


def distill_loss_backward(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, top: torch.Tensor,
                          top_logits: torch.Tensor, kept: Tuple[torch.Tensor, torch.Tensor], temperature: float = 1.0,
                          dx_dtype=None, need_dx: bool = True, need_dw: bool = True):
    """(dx [m, k] in ``dx_dtype`` (x's), dw [vocab, k] in w's type) of distill_loss; None for one not needed.

    No gradient reaches the teacher's logits."""
    heat = _heat(temperature)
    x, ldx, w, ldw = _pair(x, w)
    (m, k), vocab, d = x.shape, w.shape[0], x.device
    items, bits, logits, ld, t = _lists(top, top_logits, m)
    dloss, lse, scores = _floats(dloss, (m,), "dloss"), _floats(kept[0], (m,), "lse"), _floats(kept[1], (m, t), "scores")
    _here(x, w, items, logits, dloss, lse, scores)
    code, dtype = _dtype_code(x.dtype if dx_dtype is None else dx_dtype), _dtype_code(x.dtype)
    dx = torch.empty((m, k), dtype=_TORCH_DTYPE[code], device=d) if need_dx else None
    dw = torch.empty((vocab, k), dtype=x.dtype, device=d) if need_dw else None
    nb = lib().distill_loss_backward_workspace_bytes(m, vocab, k, t, dtype)
    ws = _scratch("softmax_loss_backward", nb, d)
    _check(lib().distill_loss_backward(_ptr(dloss), _ptr(x), ldx, _ptr(w), ldw, dtype, m, vocab, k, _ptr(items), bits,
                                       _ptr(logits), _dtype_code(logits.dtype), ld, t, _ptr(lse), _ptr(scores), heat,
                                       _ptr(dx), code, _ptr(dw), _ptr(ws), nb, _stream()))
    return dx, dw
