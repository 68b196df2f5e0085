"""Dense operators on looked-up rows: per-group norms and matrix products.

Rows of a lookup belong to groups (the feature table of each row, or the
expert a router chose for it).  :func:`group_rows` makes the plan of which
rows belong to which group; the norms and products below take it and leave
the rows where they are.  Every function is one asynchronous library call (or
two) on the current stream; gradients are functions of their own, as the
library's backward calls are.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple, Union

import torch

from ._binding import _TORCH_DTYPE, _check, _dev, _dtype_code, _ptr, _stream, _workspace, lib

_FMT = {"i8": 0, "e4m3": 1}
_KIND = {"rms": 0, "layer": 1}
_ACT = {"none": 0, "sigmoid": 1, "silu": 2}
_INT32 = torch.int32
_INT_MAX = 2**31 - 1          # of the library's group counts and row lengths


class RowGroups(NamedTuple):
    """Which rows belong to which of n_groups groups.

    ids int32[m]: each row's group (outside [0, n_groups): none); order
    int32[m]: rows group by group, those of no group last; offsets
    int32[n_groups + 1]: where each group starts in order."""
    ids: torch.Tensor
    order: torch.Tensor
    offsets: torch.Tensor
    n_groups: int


class Rows8(NamedTuple):
    """Rows kept in 8 bits: codes uint8[m, dim], scales uint8[m, ceil(dim / 32)],
    the format ("i8" or "e4m3") and the type the rows had."""
    codes: torch.Tensor
    scales: torch.Tensor
    fmt: str
    dtype: torch.dtype


def _scratch(tag: str, nbytes: int, device) -> torch.Tensor:
    """A call's workspace: the stream's cached one, or, into a graph being captured, one of the graph's own (the
    cached one may be replaced by a larger one while the graph lives)."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    return _workspace(tag, nbytes, device)


def _choice(table: dict, value, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {value!r}")
    return table[value]


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None, dtype=None) -> Tuple[torch.Tensor, int]:
    """A 2-D GPU tensor of f32 or bf16 and its row stride; rows may be strided, elements of a row may not."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    d, shape = t.dtype, t.shape
    if d != torch.float32 and d != torch.bfloat16:
        raise ValueError(f"{name} must be float32 or bfloat16, got {d}")
    if dtype is not None and d != dtype:
        raise ValueError(f"{name} must be {dtype}, got {d}")
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, got {len(shape)}")
    if like is not None and shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(shape)}")
    m, n = shape
    if n > _INT_MAX:
        raise ValueError(f"{name} must have rows of at most {_INT_MAX} elements, got {n}")
    ld, step = t.stride()
    if n > 1 and step != 1 or m > 1 and ld < n:
        t, ld = t.contiguous(), n
    return t, ld if m > 1 else n


def _params(weight, bias, groups, dim: int):
    """(weight, bias, n_groups) with fp32 parameters of shape [n_groups, dim] (or [dim] for one group)."""
    n = 1 if groups is None else groups.n_groups
    out = []
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            out.append(None)
            continue
        t = _dev(t, torch.float32, name)
        if tuple(t.shape) != (n, dim) and not (n == 1 and tuple(t.shape) == (dim,)):
            raise ValueError(f"{name} must have shape {(n, dim)}, got {tuple(t.shape)}")
        out.append(t)
    return out[0], out[1], n


def _index(t: Optional[torch.Tensor], n: int, name: str) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.dtype is not _INT32 or t.numel() != n or not t.is_cuda:
        raise ValueError(f"groups.{name} must be a GPU tensor of {n} int32, got {t.numel()} {t.dtype} on {t.device}")
    return t.contiguous()


def _ids(groups: Optional[RowGroups], m: int) -> Optional[torch.Tensor]:
    """Each row's group, for m rows."""
    return None if groups is None else _index(groups.ids, m, "ids")


def _plan(groups: Optional[RowGroups], m: int) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(order, offsets) of a plan for m rows."""
    if groups is None:
        return None, None
    return _index(groups.order, m, "order"), _index(groups.offsets, groups.n_groups + 1, "offsets")


def _new_rows8(m: int, dim: int, fmt: str, dtype, device) -> Rows8:
    _choice(_FMT, fmt, "format")
    return Rows8(torch.empty((m, dim), dtype=torch.uint8, device=device),
                 torch.empty((m, (dim + 31) // 32), dtype=torch.uint8, device=device), fmt, dtype)


def _check_rows8(r: Rows8, name: str) -> Rows8:
    _choice(_FMT, r.fmt, "format")
    if r.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name}.dtype must be float32 or bfloat16, got {r.dtype}")
    codes, scales = _dev(r.codes, torch.uint8, name + ".codes"), _dev(r.scales, torch.uint8, name + ".scales")
    if codes.dim() != 2 or tuple(scales.shape) != (codes.shape[0], (codes.shape[1] + 31) // 32):
        raise ValueError(f"{name}: scales must have shape [rows, ceil(dim / 32)]")
    if codes.shape[1] > _INT_MAX:
        raise ValueError(f"{name} must have rows of at most {_INT_MAX} elements, got {codes.shape[1]}")
    return Rows8(codes, scales, r.fmt, r.dtype)


def group_rows(ids: torch.Tensor, n_groups: int) -> RowGroups:
    """The plan of rows by group: a stable sort of ``ids`` (int32), rows of no group last (row_groups)."""
    if n_groups > _INT_MAX:
        raise ValueError(f"n_groups must be at most {_INT_MAX}, got {n_groups}")
    ids = _dev(ids, torch.int32, "ids").view(-1)
    m, d = ids.numel(), ids.device
    order = torch.empty(m, dtype=torch.int32, device=d)
    offsets = torch.empty(max(int(n_groups), 0) + 1, dtype=torch.int32, device=d)
    nb = lib().row_groups_workspace_bytes(m, n_groups)
    ws = _scratch("row_groups", nb, d)
    _check(lib().row_groups(_ptr(ids), m, n_groups, _ptr(order), _ptr(offsets), _ptr(ws), nb, _stream()))
    return RowGroups(ids, order, offsets, int(n_groups))


def save_rows8(x: torch.Tensor, fmt: str) -> Rows8:
    """Rows in 8 bits: blocks of 32 share a power of two, codes are integers ("i8") or e4m3 numbers (rows8_save)."""
    x, ld = _rows(x, "x")
    m, dim = x.shape
    out = _new_rows8(m, dim, fmt, x.dtype, x.device)
    _check(lib().rows8_save(_ptr(x), _dtype_code(x.dtype), ld, m, dim, _FMT[fmt], _ptr(out.codes), _ptr(out.scales),
                            _stream()))
    return out


def load_rows8(rows: Rows8, out_dtype=None) -> torch.Tensor:
    """What 8-bit rows stand for, in their own type or in ``out_dtype`` (rows8_load)."""
    rows = _check_rows8(rows, "rows")
    m, dim = rows.codes.shape
    code = _dtype_code(rows.dtype if out_dtype is None else out_dtype)
    y = torch.empty((m, dim), dtype=_TORCH_DTYPE[code], device=rows.codes.device)
    _check(lib().rows8_load(_ptr(rows.codes), _ptr(rows.scales), _FMT[rows.fmt], m, dim, _ptr(y), code, _stream()))
    return y


def norm_rows(x: Union[torch.Tensor, Rows8], weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
              groups: Optional[RowGroups] = None, kind: str = "rms", eps: float = 1e-6, out_dtype=None,
              save: Optional[str] = None):
    """A norm per row with its group's parameters (norm_rows).

    Returns (y, kept): kept is what norm_rows_backward takes, x itself, or
    with ``save`` ("i8" or "e4m3") its 8-bit copy written in the same pass.
    x may itself be Rows8 (the norm recomputed from what was kept)."""
    kind_code = _choice(_KIND, kind, "kind")
    if isinstance(x, Rows8):
        if save is not None:
            raise ValueError("x is in 8 bits already")
        x = _check_rows8(x, "x")
        src, ld, scales, fmt = x.codes, x.codes.shape[1], x.scales, _FMT[x.fmt]
    else:
        x, ld = _rows(x, "x")
        src, scales, fmt = x, None, 0
    m, dim = src.shape
    weight, bias, n = _params(weight, bias, groups, dim)
    ids = _ids(groups, m)
    code = _dtype_code(x.dtype if out_dtype is None else out_dtype)
    kept = x if save is None else _new_rows8(m, dim, save, x.dtype, src.device)
    codes, out_scales = (None, None) if save is None else (kept.codes, kept.scales)
    y = torch.empty((m, dim), dtype=_TORCH_DTYPE[code], device=src.device)
    _check(lib().norm_rows(_ptr(src), _dtype_code(x.dtype), ld, _ptr(scales), fmt, m, dim, _ptr(weight), _ptr(bias),
                           _ptr(ids), n, kind_code, eps, _ptr(y), code, _ptr(codes), _ptr(out_scales),
                           0 if save is None else _FMT[save], _stream()))
    return y, kept


def norm_rows_backward(dy: torch.Tensor, kept: Union[torch.Tensor, Rows8], weight: torch.Tensor,
                       groups: Optional[RowGroups] = None, kind: str = "rms", eps: float = 1e-6, bias: bool = False,
                       dresidual: Optional[torch.Tensor] = None):
    """(dx, dweight, dbias or None) of norm_rows at what was kept of x (norm_rows_backward).

    ``dresidual`` (of x's type) is added to dx in the same pass; dweight and
    dbias are fp32 [n_groups, dim]."""
    kind_code = _choice(_KIND, kind, "kind")
    if isinstance(kept, Rows8):
        kept = _check_rows8(kept, "kept")
        src, ldx, scales, fmt = kept.codes, kept.codes.shape[1], kept.scales, _FMT[kept.fmt]
    else:
        kept, ldx = _rows(kept, "kept")
        src, scales, fmt = kept, None, 0
    dy, ld_dy = _rows(dy, "dy", src)
    m, dim = src.shape
    res, ld_res = (None, 0) if dresidual is None else _rows(dresidual, "dresidual", src, kept.dtype)
    weight, _, n = _params(weight, None, groups, dim)
    order, offsets = _plan(groups, m)
    d = src.device
    dx = torch.empty((m, dim), dtype=kept.dtype, device=d)
    dweight = torch.empty((n, dim), dtype=torch.float32, device=d)
    dbias = torch.empty((n, dim), dtype=torch.float32, device=d) if bias else None
    nb = lib().norm_back_workspace_bytes(m, n, dim)
    ws = _scratch("norm_back", nb, d)
    _check(lib().norm_rows_backward(_ptr(dy), _dtype_code(dy.dtype), ld_dy, _ptr(src), _dtype_code(kept.dtype), ldx,
                                    _ptr(scales), fmt, _ptr(res), ld_res, m, dim, _ptr(weight), _ptr(order),
                                    _ptr(offsets), n, kind_code, eps, _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(ws),
                                    nb, _stream()))
    return dx, dweight, dbias


def norm_gate(x: torch.Tensor, z: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor,
              bias: Optional[torch.Tensor] = None, groups: Optional[RowGroups] = None, kind: str = "rms",
              eps: float = 1e-6, act: str = "silu", scale: float = 1.0, save: Optional[str] = None):
    """The end of a block: out = x + scale * act(gate) * norm(z) (norm_gate).

    Returns (out, kept_z, kept_gate): what norm_gate_backward takes, z and
    gate themselves, or with ``save`` their 8-bit copies."""
    kind_code, act_code = _choice(_KIND, kind, "kind"), _choice(_ACT, act, "act")
    x, ldx = _rows(x, "x")
    z, ldz = _rows(z, "z", x)
    gate, ldu = _rows(gate, "gate", x, z.dtype)
    m, dim = x.shape
    weight, bias, n = _params(weight, bias, groups, dim)
    ids = _ids(groups, m)
    kept_z, kept_u = z, gate
    codes = (None,) * 4
    if save is not None:
        kept_z = _new_rows8(m, dim, save, z.dtype, x.device)
        kept_u = _new_rows8(m, dim, save, z.dtype, x.device)
        codes = (kept_z.codes, kept_z.scales, kept_u.codes, kept_u.scales)
    out = torch.empty((m, dim), dtype=x.dtype, device=x.device)
    _check(lib().norm_gate(_ptr(x), _dtype_code(x.dtype), ldx, _ptr(z), ldz, _ptr(gate), ldu, _dtype_code(z.dtype), m,
                           dim, _ptr(weight), _ptr(bias), _ptr(ids), n, kind_code, eps, act_code, scale, _ptr(out),
                           *(_ptr(c) for c in codes), 0 if save is None else _FMT[save], _stream()))
    return out, kept_z, kept_u


def norm_gate_backward(dout: torch.Tensor, kept_z: Union[torch.Tensor, Rows8], kept_gate: Union[torch.Tensor, Rows8],
                       weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       groups: Optional[RowGroups] = None, kind: str = "rms", eps: float = 1e-6, act: str = "silu",
                       scale: float = 1.0):
    """(dz, dgate, dweight, dbias or None) of norm_gate at what was kept of z and gate (norm_gate_backward).

    The gradient of x is ``dout`` itself; dz and dgate have z's type."""
    kind_code, act_code = _choice(_KIND, kind, "kind"), _choice(_ACT, act, "act")
    if isinstance(kept_z, Rows8) != isinstance(kept_gate, Rows8):
        raise ValueError("z and gate are both in 8 bits or neither")
    if isinstance(kept_z, Rows8):
        kept_z, kept_gate = _check_rows8(kept_z, "kept_z"), _check_rows8(kept_gate, "kept_gate")
        if kept_z.fmt != kept_gate.fmt or kept_z.dtype != kept_gate.dtype or kept_z.codes.shape != kept_gate.codes.shape:
            raise ValueError("z and gate must be kept in one format, type and shape")
        z, u, fmt = kept_z.codes, kept_gate.codes, _FMT[kept_z.fmt]
        ldz = ldu = z.shape[1]
        zs, us = kept_z.scales, kept_gate.scales
    else:
        z, ldz = _rows(kept_z, "kept_z")
        u, ldu = _rows(kept_gate, "kept_gate", z, z.dtype)
        zs = us = None
        fmt = 0
    dtype = kept_z.dtype
    dout, ld = _rows(dout, "dout", z)
    m, dim = z.shape
    weight, bias, n = _params(weight, bias, groups, dim)
    order, offsets = _plan(groups, m)
    d = z.device
    dz = torch.empty((m, dim), dtype=dtype, device=d)
    du = torch.empty((m, dim), dtype=dtype, device=d)
    dweight = torch.empty((n, dim), dtype=torch.float32, device=d)
    dbias = None if bias is None else torch.empty((n, dim), dtype=torch.float32, device=d)
    nb = lib().norm_back_workspace_bytes(m, n, dim)
    ws = _scratch("norm_back", nb, d)
    _check(lib().norm_gate_backward(_ptr(dout), _dtype_code(dout.dtype), ld, _ptr(z), ldz, _ptr(zs), _ptr(u), ldu,
                                    _ptr(us), _dtype_code(dtype), fmt, m, dim, _ptr(weight), _ptr(bias), _ptr(order),
                                    _ptr(offsets), n, kind_code, eps, act_code, scale, _ptr(dz), _ptr(du),
                                    _ptr(dweight), _ptr(dbias), _ptr(ws), nb, _stream()))
    return dz, du, dweight, dbias


def _weights(w: torch.Tensor, groups: Optional[RowGroups], dtype) -> Tuple[torch.Tensor, int]:
    w = _dev(w, dtype, "w")
    n = 1 if groups is None else groups.n_groups
    if w.dim() == 2 and n == 1:
        w = w.unsqueeze(0)
    if w.dim() != 3 or w.shape[0] != n:
        raise ValueError(f"w must have shape [{n}, n, k], got {tuple(w.shape)}")
    if w.shape[1] > _INT_MAX:
        raise ValueError(f"w must have at most {_INT_MAX} outputs, got {w.shape[1]}")
    return w, n


def grouped_mm(x: torch.Tensor, w: torch.Tensor, groups: Optional[RowGroups] = None, out_dtype=None) -> torch.Tensor:
    """y[i] = w[g] @ x[i], g the group of row i; zeros for rows of no group (grouped_mm).

    x [m, k] and w [n_groups, n, k] of one type (w [n, k] without groups);
    y [m, n] in ``out_dtype`` (x's)."""
    x, ldx = _rows(x, "x")
    w, g = _weights(w, groups, x.dtype)
    m, k = x.shape
    n = w.shape[1]
    if w.shape[2] != k:
        raise ValueError(f"x has rows of {k}, w of {w.shape[2]}")
    order, offsets = _plan(groups, m)
    code = _dtype_code(x.dtype if out_dtype is None else out_dtype)
    y = torch.empty((m, n), dtype=_TORCH_DTYPE[code], device=x.device)
    _check(lib().grouped_mm(_ptr(x), ldx, _ptr(w), _dtype_code(x.dtype), m, n, k, _ptr(order), _ptr(offsets), g,
                            _ptr(y), code, _stream()))
    return y


def grouped_mm_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, groups: Optional[RowGroups] = None,
                        dx_dtype=None, need_dx: bool = True, need_dw: bool = True):
    """(dx [m, k] in ``dx_dtype`` (dy's), dw fp32 [n_groups, n, k]) of grouped_mm; None for one not needed."""
    x, ldx = _rows(x, "x")
    dy, ld_dy = _rows(dy, "dy", dtype=x.dtype)
    w, g = _weights(w, groups, x.dtype)
    m, k = x.shape
    n = w.shape[1]
    if w.shape[2] != k or tuple(dy.shape) != (m, n):
        raise ValueError(f"dy {tuple(dy.shape)}, x {tuple(x.shape)} and w {tuple(w.shape)} do not fit")
    order, offsets = _plan(groups, m)
    code = _dtype_code(dy.dtype if dx_dtype is None else dx_dtype)
    d = x.device
    dx = torch.empty((m, k), dtype=_TORCH_DTYPE[code], device=d) if need_dx else None
    dw = torch.empty((g, n, k), dtype=torch.float32, device=d) if need_dw else None
    nb = lib().grouped_mm_backward_workspace_bytes(m, g, n, k) if need_dw else 0
    ws = _scratch("grouped_mm_backward", nb, d) if need_dw else None
    _check(lib().grouped_mm_backward(_ptr(dy), ld_dy, _ptr(x), ldx, _ptr(w), _dtype_code(x.dtype), m, n, k, _ptr(order),
                                     _ptr(offsets), g, _ptr(dx), code, _ptr(dw), _ptr(ws), nb, _stream()))
    return dx, dw
