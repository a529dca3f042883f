"""Binding of include/moe_adapter.h: low-rank adapters of many requests beside
a shared projection, forward and backward.  Checks and marshalling only, as in
dispatch.py; x, dy, add and out may be row-strided views (last stride 1)."""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import lib
from .dispatch import _F32, _I32, _check, _ptr, _rows_dtype, _run


_ADAPTERS = struct.Struct("@PPPPiiiii").pack


def _check_rows(name, t, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape or t.device != dev or (t.numel() and t.stride(1) != 1):
        raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)} on {dev} with contiguous rows is needed, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.stride(0) if shape[0] > 1 else max(shape[1], 8)


def _adapters(x, a, b, scale, ranks, ids, order):
    code = _rows_dtype("x", x)
    dev = x.device
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a [n][R][K] and b [n][N][R] are needed")
    n, R, K = a.shape
    N = b.shape[1]
    T = x.shape[0]
    _check("a", a, x.dtype, (n, R, K), dev)
    _check("b", b, x.dtype, (n, N, R), dev)
    _check("scale", scale, _F32, (n,), dev)
    if ranks is not None:
        _check("ranks", ranks, _I32, (n,), dev)
    _check("ids", ids, _I32, (T,), dev)
    off = pairs = None
    if order is not None:
        off, pairs = order["offsets"], order["pairs"]
        _check("order: offsets", off, _I32, (n + 1,), dev)
        _check("order: pairs", pairs, _I32, (T,), dev)
    # a moe_adapters_t
    d = _ADAPTERS(a.data_ptr(), b.data_ptr(), scale.data_ptr(), 0 if ranks is None else ranks.data_ptr(), n, K, N, R, code)
    ws = torch.empty(lib().moe_adapter_workspace_bytes(d, T), dtype=torch.uint8, device=dev)
    return d, dev, T, n, K, N, R, off, pairs, ws


def moe_adapter_forward(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor, scale: torch.Tensor,
                        ranks: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None, order=None,
                        out: Optional[torch.Tensor] = None, save_u: bool = False, stream=None):
    """y[t] = add[t] + scale[i] * b[i] @ (a[i] @ x[t]) with i = ids[t] (none:
    just add[t], or zeros).  x [T][K], a [n][R][K], b [n][N][R]; ids int32 [T];
    ranks int32 [n]: each adapter's rank where below R; add [T][N] (may be
    `out`); order: moe_sort(ids[:, None], n) where the caller has it.
    save_u: returns (y, u) with u = a[i] @ x[t] fp32 [T][R] for the backward."""
    d, dev, T, n, K, N, R, off, pairs, ws = _adapters(x, a, b, scale, ranks, ids, order)
    ldx = _check_rows("x", x, x.dtype, (T, K), dev)
    ldadd = 0 if add is None else _check_rows("add", add, x.dtype, (T, N), dev)
    made = [ws]
    if out is None:
        out = x.new_empty((T, N))
        made.append(out)
    ldy = _check_rows("out", out, x.dtype, (T, N), dev)
    u = scale.new_empty((T, R)) if save_u else None
    if save_u:
        made.append(u)
    _run(lib().moe_adapter_forward, dev, stream, made, d, x.data_ptr(), ldx, T, ids.data_ptr(),
         _ptr(off), _ptr(pairs), _ptr(add), ldadd, out.data_ptr(), ldy, _ptr(u), ws.data_ptr(), ws.numel())
    return (out, u) if save_u else out


def moe_adapter_backward(dy: torch.Tensor, x: torch.Tensor, u: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                         ids: torch.Tensor, scale: torch.Tensor, ranks: Optional[torch.Tensor] = None,
                         add: Optional[torch.Tensor] = None, order=None, need_dx: bool = True, stream=None):
    """(dx [T][K] or None, da fp32 [n][R][K], db fp32 [n][N][R]) for dy [T][N];
    u from the forward call; add [T][K] is added to dx."""
    d, dev, T, n, K, N, R, off, pairs, ws = _adapters(x, a, b, scale, ranks, ids, order)
    ldx = _check_rows("x", x, x.dtype, (T, K), dev)
    lddy = _check_rows("dy", dy, x.dtype, (T, N), dev)
    _check("u", u, _F32, (T, R), dev)
    ldadd = 0 if add is None else _check_rows("add", add, x.dtype, (T, K), dev)
    if add is not None and not need_dx:
        raise ValueError("add: there is no dx to add it to")
    dx = x.new_empty((T, K)) if need_dx else None
    da = scale.new_empty((n, R, K))
    db = scale.new_empty((n, N, R))
    _run(lib().moe_adapter_backward, dev, stream, [ws, da, db] + ([dx] if need_dx else []), d,
         dy.data_ptr(), lddy, x.data_ptr(), ldx, u.data_ptr(), T, ids.data_ptr(), _ptr(off), _ptr(pairs), _ptr(add),
         ldadd, _ptr(dx), K, da.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel())
    return dx, da, db
