"""Binding of include/moe_dispatch.h: tokens laid out by expert and back, the
gradients of that path and of the router's weights.

Argument checks and marshalling only; each function carries the name of its C
entry point and runs on the tensors' device and (unless `stream` is given) on
that device's current stream.  Tensors of the wrong type, shape or device, or
not contiguous, raise ValueError; what the library refuses raises MoeError.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import MOE_OK, MoeError, lib

MOE_T_F16, MOE_T_BF16, MOE_T_F32 = 0, 1, 2
_DTYPES = {torch.float16: MOE_T_F16, torch.bfloat16: MOE_T_BF16, torch.float32: MOE_T_F32}
_I32, _F32 = torch.int32, torch.float32


def _check(name, t, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {dev} is needed, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _rows_dtype(name, t, dims=2):
    if t.dim() != dims or t.device.type != "cuda":
        raise ValueError(f"{name}: a {dims}-dimensional tensor on a GPU is needed, got {tuple(t.shape)} on {t.device}")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: float16, bfloat16 or float32 rows are needed, got {t.dtype}")
    return code


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The raw handle and device index, without the objects that torch.cuda wraps
# around them: a small call's time is mostly its host side.
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _run(fn, dev, stream, made, *args):
    """Calls a C entry point on `dev` and `stream`; `made` are the tensors
    allocated here, kept from reuse until that stream has passed the call."""
    index = dev.index
    handle = _current_stream(index)
    if stream is not None:
        given = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if given != handle:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(given, device=dev)
            s.wait_stream(torch.cuda.current_stream(dev))  # the allocator may hand out memory still in use there
            for t in made:
                if t is not None:
                    t.record_stream(s)
            handle = given
    if index == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != MOE_OK:
        raise MoeError(rc, fn.__name__)


def moe_sort_rows(T: int, k: int, n_experts: int, align: int = 1) -> int:
    """Rows of the expert-sorted buffers."""
    n = int(lib().moe_sort_rows(T, k, n_experts, align))
    if n < 0:  # (the size query has no status; the sort checks the shape before anything else)
        raise MoeError(lib().moe_sort(None, T, k, n_experts, align, None, None, None, None, 0, None), "moe_sort_rows")
    return n


def _sort_buffers(topk_idx, n_experts, align):
    if topk_idx.dim() != 2 or topk_idx.device.type != "cuda":
        raise ValueError(f"topk_idx: an int32 tensor [T][k] on a GPU is needed, got {tuple(topk_idx.shape)} on "
                         f"{topk_idx.device}")
    T, k = topk_idx.shape
    dev = topk_idx.device
    _check("topk_idx", topk_idx, _I32, (T, k), dev)
    rows = moe_sort_rows(T, k, n_experts, align)
    offsets, pairs, pos = topk_idx.new_empty(n_experts + 1), topk_idx.new_empty(rows), torch.empty_like(topk_idx)
    need = lib().moe_sort_workspace_bytes(T, k, n_experts)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    return T, k, dev, rows, offsets, pairs, pos, ws


def moe_sort(topk_idx: torch.Tensor, n_experts: int, align: int = 1, stream=None):
    """Slots of topk_idx (int32 [T][k]; entries outside [0, n_experts) are
    dropped) sorted by expert: dict(offsets [E + 1], pairs [rows], pos [T][k])."""
    T, k, dev, _, offsets, pairs, pos, ws = _sort_buffers(topk_idx, n_experts, align)
    _run(lib().moe_sort, dev, stream, (offsets, pairs, pos, ws), topk_idx.data_ptr(), T, k, n_experts, align,
         offsets.data_ptr(), pairs.data_ptr(), pos.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return dict(offsets=offsets, pairs=pairs, pos=pos)


def moe_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, n_experts: int, align: int = 1, stream=None):
    """moe_sort, and xs [rows][H]: x[t] in the row of each kept slot, zeros in
    the others.  dict(xs, offsets, pairs, pos)."""
    code = _rows_dtype("x", x)
    T, k, dev, rows, offsets, pairs, pos, ws = _sort_buffers(topk_idx, n_experts, align)
    H = x.shape[1]
    _check("x", x, x.dtype, (T, H), dev)
    xs = x.new_empty((rows, H))
    _run(lib().moe_dispatch, dev, stream, (xs, offsets, pairs, pos, ws), x.data_ptr(), code, T, H,
         topk_idx.data_ptr(), k, n_experts, align, xs.data_ptr(), offsets.data_ptr(), pairs.data_ptr(),
         pos.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return dict(xs=xs, offsets=offsets, pairs=pairs, pos=pos)


def _gather_args(name, o, pos, add, out):
    code = _rows_dtype(name, o)
    dev = o.device
    if pos.dim() != 2:
        raise ValueError(f"pos: an int32 tensor [T][k] is needed, got {tuple(pos.shape)}")
    (rows, H), (T, k) = o.shape, pos.shape
    _check(name, o, o.dtype, (rows, H), dev)
    _check("pos", pos, _I32, (T, k), dev)
    if add is not None:
        _check("add", add, o.dtype, (T, H), dev)
    made = ()
    if out is None:
        out = o.new_empty((T, H))
        made = (out,)
    else:
        _check("out", out, o.dtype, (T, H), dev)
    return code, dev, rows, H, T, k, out, made


def moe_dispatch_backward(dxs: torch.Tensor, pos: torch.Tensor, add: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dx[t] = add[t] + sum_j dxs[pos[t][j]] (`add` may be `out`)."""
    code, dev, rows, H, T, k, out, made = _gather_args("dxs", dxs, pos, add, out)
    _run(lib().moe_dispatch_backward, dev, stream, made, dxs.data_ptr(), code, rows, H, pos.data_ptr(), T, k,
         _ptr(add), out.data_ptr())
    return out


def moe_combine(o: torch.Tensor, topk_w: torch.Tensor, pos: torch.Tensor, add: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = add[t] + sum_j topk_w[t][j] * o[pos[t][j]] (`add` may be `out`)."""
    code, dev, rows, H, T, k, out, made = _gather_args("o", o, pos, add, out)
    _check("topk_w", topk_w, _F32, (T, k), dev)
    _run(lib().moe_combine, dev, stream, made, o.data_ptr(), code, rows, H, topk_w.data_ptr(), pos.data_ptr(), T, k,
         _ptr(add), out.data_ptr())
    return out


def moe_combine_backward(dy: torch.Tensor, o: torch.Tensor, topk_w: torch.Tensor, pos: torch.Tensor,
                         pairs: torch.Tensor, stream=None):
    """(d_o [rows][H], dw fp32 [T][k]) for dy [T][H]; rows without a slot get zeros."""
    code = _rows_dtype("o", o)
    dev = o.device
    if pos.dim() != 2:
        raise ValueError(f"pos: an int32 tensor [T][k] is needed, got {tuple(pos.shape)}")
    (rows, H), (T, k) = o.shape, pos.shape
    _check("o", o, o.dtype, (rows, H), dev)
    _check("dy", dy, o.dtype, (T, H), dev)
    _check("topk_w", topk_w, _F32, (T, k), dev)
    _check("pos", pos, _I32, (T, k), dev)
    _check("pairs", pairs, _I32, (rows,), dev)
    d_o = torch.empty_like(o)
    dw = torch.empty_like(topk_w)
    _run(lib().moe_combine_backward, dev, stream, (d_o, dw), dy.data_ptr(), o.data_ptr(), code, rows, H,
         topk_w.data_ptr(), pos.data_ptr(), pairs.data_ptr(), T, k, d_o.data_ptr(), dw.data_ptr())
    return d_o, dw


def moe_route_backward(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
                       topk_idx: torch.Tensor, dw: torch.Tensor, offsets: torch.Tensor, pairs: torch.Tensor,
                       add: Optional[torch.Tensor] = None, stream=None):
    """(dx [T][H], d_router_w fp32 [E][H], d_router_b fp32 [E]) for the
    gradient dw of moe_route's topk_w; offsets and pairs from moe_sort (or
    moe_dispatch) of topk_idx; add [T][H] is added to dx."""
    code = _rows_dtype("x", x)
    dev = x.device
    if topk_idx.dim() != 2 or router_w.dim() != 2 or pairs.dim() != 1:
        raise ValueError("topk_idx [T][k], router_w [E][H] and pairs [rows] are needed")
    T, k = topk_idx.shape
    E, H = router_w.shape
    rows = pairs.shape[0]
    _check("x", x, x.dtype, (T, H), dev)
    _check("router_w", router_w, _F32, (E, H), dev)
    if router_b is not None:
        _check("router_b", router_b, _F32, (E,), dev)
    _check("topk_idx", topk_idx, _I32, (T, k), dev)
    _check("dw", dw, _F32, (T, k), dev)
    _check("offsets", offsets, _I32, (E + 1,), dev)
    _check("pairs", pairs, _I32, (rows,), dev)
    if add is not None:
        _check("add", add, x.dtype, (T, H), dev)
    dx, dwr, db = torch.empty_like(x), torch.empty_like(router_w), router_w.new_empty(E)
    ws = torch.empty(lib().moe_route_backward_workspace_bytes(T, k, E, H, rows), dtype=torch.uint8, device=dev)
    _run(lib().moe_route_backward, dev, stream, (dx, dwr, db, ws), x.data_ptr(), code, T, H, E, k,
         router_w.data_ptr(), _ptr(router_b), topk_idx.data_ptr(), dw.data_ptr(), offsets.data_ptr(),
         pairs.data_ptr(), rows, _ptr(add), dx.data_ptr(), dwr.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel())
    return dx, dwr, db
