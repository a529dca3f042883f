"""Binding of include/moe_w4.h: products of rows with frozen 4-bit weights that
have group scales, of one matrix or one per expert, and the gradient of the rows.
Checks and marshalling only, as in dispatch.py; x, dy, add and out may be
row-strided views (last stride 1)."""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import lib
from .adapter import _check_rows
from .dispatch import _I32, MOE_T_F32, _check, _ptr, _rows_dtype, _run

_DIMS = struct.Struct("@iiiiii").pack


class W4Weights:
    """n packed matrices [N][K] (moe_w4_pack): `packed` uint8, `shape` (n, N, K),
    `group` columns per scale, `zeros` whether there are zero points, and the
    rows' and scales' `dtype`."""

    def __init__(self, packed: torch.Tensor, n: int, N: int, K: int, group: int, zeros: bool, dtype: torch.dtype, code: int):
        self.packed, self.shape, self.group, self.zeros, self.dtype = packed, (n, N, K), group, zeros, dtype
        self.dims = _DIMS(n, N, K, group, int(zeros), code)  # a moe_w4_dims_t


def moe_w4_pack(q: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None, stream=None) -> W4Weights:
    """Packs q uint8 [n][N][K / 2] (int4 codes, column 2j in the low nibble of byte
    j), scales [n][N][K / group] (their type is the rows') and zeros int8 of the
    scales' shape, or None; one matrix may come without its first dimension."""
    if q.dim() == 2:
        q, scales, zeros = q[None], scales[None], None if zeros is None else zeros[None]
    if q.dim() != 3 or scales.dim() != 3 or not scales.shape[2] or 2 * q.shape[2] % scales.shape[2]:
        raise ValueError(f"q [n][N][K / 2] and scales [n][N][K / group] are needed, got {tuple(q.shape)} and {tuple(scales.shape)}")
    code = _rows_dtype("scales", scales, 3)
    if code == MOE_T_F32:
        raise ValueError("scales: float16 or bfloat16 is needed")
    (n, N, half), dev = q.shape, scales.device
    shape = (n, N, scales.shape[2])
    _check("q", q, torch.uint8, (n, N, half), dev)
    _check("scales", scales, scales.dtype, shape, dev)
    if zeros is not None:
        _check("zeros", zeros, torch.int8, shape, dev)
    group = 2 * half // shape[2]
    dims = _DIMS(n, N, 2 * half, group, int(zeros is not None), code)
    # (the size query has no status; the call checks the shape before anything else)
    packed = torch.empty(lib().moe_w4_packed_bytes(dims), dtype=torch.uint8, device=dev)
    _run(lib().moe_w4_pack, dev, stream, (packed,), dims, q.data_ptr(), scales.data_ptr(), _ptr(zeros), packed.data_ptr())
    return W4Weights(packed, n, N, 2 * half, group, zeros is not None, scales.dtype, code)


def moe_w4_unpack(w: W4Weights, stream=None):
    """(q, scales, zeros or None) of packed weights."""
    n, N, K = w.shape
    q = w.packed.new_empty((n, N, K // 2))
    scales = torch.empty((n, N, K // w.group), dtype=w.dtype, device=w.packed.device)
    zeros = torch.empty(scales.shape, dtype=torch.int8, device=w.packed.device) if w.zeros else None
    _run(lib().moe_w4_unpack, w.packed.device, stream, (q, scales, zeros), w.dims, w.packed.data_ptr(), q.data_ptr(),
         scales.data_ptr(), _ptr(zeros))
    return q, scales, zeros


def moe_w4_few_rows(w: W4Weights, T: int) -> bool:
    """Whether moe_w4_forward on T rows takes the path for few rows."""
    return bool(lib().moe_w4_few_rows(w.dims, T))


def _product(fn, backward, name, x, w, into, width, offsets, add, out, stream):
    _rows_dtype(name, x)
    n, dev, T = w.shape[0], x.device, x.shape[0]
    ldx = _check_rows(name, x, w.dtype, (T, into), dev)
    if w.packed.device != dev:
        raise ValueError(f"w: packed weights on {dev} are needed, got {w.packed.device}")
    if offsets is not None:
        _check("offsets", offsets, _I32, (n + 1,), dev)
    elif n != 1:
        raise ValueError(f"offsets: int32 [{n + 1}] are needed for {n} matrices")
    ldadd = 0 if add is None else _check_rows("add", add, w.dtype, (T, width), dev)
    made = []
    if out is None:
        out = x.new_empty((T, width))
        made.append(out)
    ldy = _check_rows("out", out, w.dtype, (T, width), dev)
    need = lib().moe_w4_workspace_bytes(w.dims, T, backward)
    ws = None
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        made.append(ws)
    _run(fn, dev, stream, made, w.dims, w.packed.data_ptr(), x.data_ptr(), ldx, T, _ptr(offsets), _ptr(add), ldadd,
         out.data_ptr(), ldy, _ptr(ws), need)
    return out


def moe_w4_forward(x: torch.Tensor, w: W4Weights, offsets: Optional[torch.Tensor] = None,
                   add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = add[t] + W_e @ x[t], x [T][K]; rows offsets[e] .. offsets[e + 1] - 1
    (int32 [n + 1], as moe_dispatch gives them) use matrix e, rows outside every
    group get add[t] or zeros; `add` may be `out`, which must not share memory with `x`."""
    return _product(lib().moe_w4_forward, 0, "x", x, w, w.shape[2], w.shape[1], offsets, add, out, stream)


def moe_w4_backward(dy: torch.Tensor, w: W4Weights, offsets: Optional[torch.Tensor] = None,
                    add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dx[t] = add[t] + W_e.T @ dy[t], dy [T][N]: the gradient of moe_w4_forward's rows;
    `add` and `out` as there."""
    return _product(lib().moe_w4_backward, 1, "dy", dy, w, w.shape[1], w.shape[2], offsets, add, out, stream)
