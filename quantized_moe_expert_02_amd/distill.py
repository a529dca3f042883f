"""Binding of include/moe_distill.h: the divergence of logits from a teacher's top
logits, and its gradient.  Checks and marshalling only, as in dispatch.py; logits
and their gradient may be row-strided views (last stride 1) of any alignment."""
from __future__ import annotations

from typing import Optional

import torch

from . import lib
from .dispatch import _F32, _I32, _check, _ptr, _rows_dtype, _run


def _logits(name, t, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape or t.device != dev or (t.numel() and t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)} on {dev} with contiguous rows is needed, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _teacher(logits, ids, teacher):
    code = _rows_dtype("logits", logits)
    (T, V), dev = logits.shape, logits.device
    if ids.dim() != 2:
        raise ValueError(f"ids: an int32 tensor [T][k] is needed, got {tuple(ids.shape)}")
    k = ids.shape[1]
    _check("ids", ids, _I32, (T, k), dev)
    _check("teacher", teacher, _F32, (T, k), dev)
    return code, T, V, k, dev, _logits("logits", logits, logits.dtype, (T, V), dev)


def moe_distill_forward(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, temperature: float = 1.0,
                        stream=None):
    """(loss fp32 [T], stats fp32 [T][2]) of logits [T][V] for the teacher's logits
    `teacher` fp32 [T][k] at the columns `ids` int32 [T][k] (values outside [0, V):
    no entry; a row without entries has loss 0): sum_j p_j (log p_j - log q[ids_j])
    with p and q the softmax of teacher / temperature over the row's entries and
    of logits / temperature.  stats: the largest logit and log sum exp((z - it) /
    temperature), which the backward call takes."""
    code, T, V, k, dev, ld = _teacher(logits, ids, teacher)
    loss, stats = teacher.new_empty(T), teacher.new_empty((T, 2))
    need = lib().moe_distill_workspace_bytes(T, V, code)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _run(lib().moe_distill_forward, dev, stream, (loss, stats, ws), logits.data_ptr(), code, ld, T, V, ids.data_ptr(),
         teacher.data_ptr(), k, temperature, loss.data_ptr(), stats.data_ptr(), _ptr(ws), need)
    return loss, stats


def moe_distill_backward(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, stats: torch.Tensor,
                         dloss: torch.Tensor, temperature: float = 1.0, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """dlogits [T][V] for dloss fp32 [T]; stats from the forward call; `out` may be
    `logits`, whose values are then replaced, but must not share memory with it otherwise."""
    code, T, V, k, dev, ld = _teacher(logits, ids, teacher)
    _check("stats", stats, _F32, (T, 2), dev)
    _check("dloss", dloss, _F32, (T,), dev)
    made = ()
    if out is None:
        out = logits.new_empty((T, V))
        made = (out,)
    ldo = _logits("out", out, logits.dtype, (T, V), dev)
    _run(lib().moe_distill_backward, dev, stream, made, logits.data_ptr(), code, ld, T, V, ids.data_ptr(),
         teacher.data_ptr(), k, temperature, stats.data_ptr(), dloss.data_ptr(), out.data_ptr(), ldo)
    return out
