"""Python binding of the MI355X quantised MoE FFN layer library (libmoe_w4a16.so).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  The
functions carry the names of the C entry points declared in
include/moe_w4a16.h.  If the built library is missing, importing the binding
succeeds but every call raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_w4a16.so")

MOE_OK, MOE_E_INVAL, MOE_E_UNSUPPORTED, MOE_E_WORKSPACE, MOE_E_HIP = 0, -1, -2, -3, -4
MOE_W_INT4_ROW, MOE_W_E2M1_B16, MOE_W_INT8_ROW, MOE_W_INT2_ROW = 0, 1, 2, 3
_CODE_BITS = {MOE_W_INT4_ROW: 4, MOE_W_E2M1_B16: 4, MOE_W_INT8_ROW: 8, MOE_W_INT2_ROW: 2}

EXPORTS = ("moe_packed_bytes", "moe_workspace_bytes", "moe_workspace_sync_bytes", "moe_pack", "moe_unpack",
           "moe_route", "moe_w4a16_forward", "moe_w4a16_forward_profiled", "moe_w4a16_forward_noalloc",
           "moe_decode_max_tokens", "moe_step_graph_create", "moe_step_graph_launch", "moe_step_graph_destroy",
           "moe_probe_stream_read", "moe_probe_mfma",
           "moe_status_string", "moe_tier_create", "moe_tier_destroy", "moe_tier_use", "moe_tier_prefetch",
           "moe_tier_slot", "moe_tier_stats", "moe_tier_sync",
           "moe_sort_rows", "moe_sort_workspace_bytes", "moe_sort", "moe_dispatch", "moe_dispatch_backward",
           "moe_combine", "moe_combine_backward", "moe_route_backward_workspace_bytes", "moe_route_backward",
           "moe_adapter_workspace_bytes", "moe_adapter_forward", "moe_adapter_backward",
           "moe_w4_packed_bytes", "moe_w4_pack", "moe_w4_unpack", "moe_w4_few_rows", "moe_w4_workspace_bytes",
           "moe_w4_forward", "moe_w4_backward", "moe_distill_workspace_bytes", "moe_distill_forward",
           "moe_distill_backward")
MOE_TIER_LRU, MOE_TIER_HOT = 0, 1
MOE_NOALLOC_SCRATCH_BYTES = 32 << 20  # include/moe_w4a16.h
MOE_STEP_GRAPH_MAX_LAYERS = 4096  # include/moe_w4a16.h


class MoeDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("has_shared", ctypes.c_int32), ("wfmt", ctypes.c_int32),
                ("top_p", ctypes.c_float)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_void_p), ("shared", ctypes.c_void_p), ("router_w", ctypes.c_void_p),
                ("router_b", ctypes.c_void_p)]


class MoeTierStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_int64), ("misses", ctypes.c_int64), ("promotions", ctypes.c_int64),
                ("evictions", ctypes.c_int64), ("prefetched", ctypes.c_int64), ("bytes_promoted", ctypes.c_int64)]


class MoeAdapters(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("n", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("R", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {moe_status_string(code)} ({code})")


_lib = None


def lib():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with quantized_moe_expert_02_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        D = ctypes.POINTER(MoeDims)
        W = ctypes.POINTER(MoeWeights)
        L.moe_packed_bytes.argtypes = [D]
        L.moe_packed_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [D, i32]
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_sync_bytes.argtypes = [D]
        L.moe_workspace_sync_bytes.restype = sz
        L.moe_pack.argtypes = [D, P, P, P, P, P, P, P, P, P]
        L.moe_pack.restype = ctypes.c_int
        L.moe_unpack.argtypes = [D, P, P, P, P, P, P, P, P, P]
        L.moe_unpack.restype = ctypes.c_int
        L.moe_route.argtypes = [D, W, P, i32, P, P, P, P, P, P, P, sz, P]
        L.moe_route.restype = ctypes.c_int
        L.moe_w4a16_forward.argtypes = [D, W, P, i32, P, P, P, P, sz, P]
        L.moe_w4a16_forward.restype = ctypes.c_int
        L.moe_w4a16_forward_profiled.argtypes = [D, W, P, i32, P, P, P, P, sz, P, P, i32]
        L.moe_w4a16_forward_profiled.restype = ctypes.c_int
        L.moe_w4a16_forward_noalloc.argtypes = [D, W, P, i32, P, P, P, P]
        L.moe_w4a16_forward_noalloc.restype = ctypes.c_int
        L.moe_decode_max_tokens.restype = i32
        L.moe_step_graph_create.argtypes = [D, i32, W, P, i32, P, P, sz, ctypes.POINTER(P)]
        L.moe_step_graph_create.restype = ctypes.c_int
        L.moe_step_graph_launch.argtypes = [P, P]
        L.moe_step_graph_launch.restype = ctypes.c_int
        L.moe_step_graph_destroy.argtypes = [P]
        L.moe_step_graph_destroy.restype = ctypes.c_int
        L.moe_probe_stream_read.argtypes = [P, sz, P, i32, P]
        L.moe_probe_stream_read.restype = ctypes.c_int
        L.moe_probe_mfma.argtypes = [P, i32, i32, P]
        L.moe_probe_mfma.restype = ctypes.c_int
        L.moe_tier_create.argtypes = [D, i32, P, P, i32, P, P, i32, ctypes.POINTER(P)]
        L.moe_tier_create.restype = ctypes.c_int
        L.moe_tier_destroy.argtypes = [P]
        L.moe_tier_destroy.restype = ctypes.c_int
        L.moe_tier_use.argtypes = [P, i32, P, i32, P]
        L.moe_tier_use.restype = ctypes.c_int
        L.moe_tier_prefetch.argtypes = [P, i32, P, i32, P]
        L.moe_tier_prefetch.restype = ctypes.c_int
        L.moe_tier_slot.argtypes = [P, i32, i32]
        L.moe_tier_slot.restype = i32
        L.moe_tier_stats.argtypes = [P, ctypes.POINTER(MoeTierStats)]
        L.moe_tier_stats.restype = ctypes.c_int
        L.moe_tier_sync.argtypes = [P, P]
        L.moe_tier_sync.restype = ctypes.c_int
        i64 = ctypes.c_int64
        A = P  # const moe_adapters_t*: a MoeAdapters by reference, or its bytes
        L.moe_sort_rows.argtypes = [i32, i32, i32, i32]
        L.moe_sort_rows.restype = i64
        L.moe_sort_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_sort_workspace_bytes.restype = sz
        L.moe_sort.argtypes = [P, i32, i32, i32, i32, P, P, P, P, sz, P]
        L.moe_dispatch.argtypes = [P, i32, i32, i32, P, i32, i32, i32, P, P, P, P, P, sz, P]
        L.moe_dispatch_backward.argtypes = [P, i32, i32, i32, P, i32, i32, P, P, P]
        L.moe_combine.argtypes = [P, i32, i32, i32, P, P, i32, i32, P, P, P]
        L.moe_combine_backward.argtypes = [P, P, i32, i32, i32, P, P, P, i32, i32, P, P, P]
        L.moe_route_backward_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.moe_route_backward_workspace_bytes.restype = sz
        L.moe_route_backward.argtypes = [P, i32, i32, i32, i32, i32, P, P, P, P, P, P, i32, P, P, P, P, P, sz, P]
        L.moe_adapter_workspace_bytes.argtypes = [A, i32]
        L.moe_adapter_workspace_bytes.restype = sz
        L.moe_adapter_forward.argtypes = [A, P, i64, i32, P, P, P, P, i64, P, i64, P, P, sz, P]
        L.moe_adapter_backward.argtypes = [A, P, i64, P, i64, P, i32, P, P, P, P, i64, P, i64, P, P, P, sz, P]
        L.moe_w4_packed_bytes.argtypes = [P]  # const moe_w4_dims_t*: its bytes
        L.moe_w4_packed_bytes.restype = sz
        L.moe_w4_pack.argtypes = [P, P, P, P, P, P]
        L.moe_w4_unpack.argtypes = [P, P, P, P, P, P]
        L.moe_w4_few_rows.argtypes = [P, i32]
        L.moe_w4_few_rows.restype = i32
        L.moe_w4_workspace_bytes.argtypes = [P, i32, i32]
        L.moe_w4_workspace_bytes.restype = sz
        L.moe_w4_forward.argtypes = [P, P, P, i64, i32, P, P, i64, P, i64, P, sz, P]
        L.moe_w4_backward.argtypes = [P, P, P, i64, i32, P, P, i64, P, i64, P, sz, P]
        f32 = ctypes.c_float
        L.moe_distill_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_distill_workspace_bytes.restype = sz
        L.moe_distill_forward.argtypes = [P, i32, i64, i32, i32, P, P, i32, f32, P, P, P, sz, P]
        L.moe_distill_backward.argtypes = [P, i32, i64, i32, i32, P, P, i32, f32, P, P, P, i64, P]
        for n in ("moe_w4_pack", "moe_w4_unpack", "moe_w4_forward", "moe_w4_backward", "moe_distill_forward",
                  "moe_distill_backward", "moe_sort", "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
                  "moe_route_backward", "moe_adapter_forward", "moe_adapter_backward"):
            getattr(L, n).restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _dims(d) -> MoeDims:
    if isinstance(d, MoeDims):
        return d
    t = d.as_tuple() if hasattr(d, "as_tuple") else tuple(d)
    return MoeDims(*[int(v) for v in t[:6]], float(getattr(d, "top_p", t[6] if len(t) > 6 else 0.0)))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def moe_status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def moe_packed_bytes(dims) -> int:
    return int(lib().moe_packed_bytes(ctypes.byref(_dims(dims))))


def moe_workspace_bytes(dims, T: int) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(_dims(dims)), int(T)))


def moe_workspace_sync_bytes(dims) -> int:
    return int(lib().moe_workspace_sync_bytes(ctypes.byref(_dims(dims))))


def moe_decode_max_tokens() -> int:
    return int(lib().moe_decode_max_tokens())


def workspace(dims, T: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of moe_workspace_bytes(dims, T) bytes."""
    n = moe_workspace_bytes(dims, T)
    if n == 0:
        raise MoeError(MOE_E_INVAL, "moe_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_pack(dims, q_gate, s_gate, q_up, s_up, q_down, s_down, g3=None, out=None, stream=None) -> torch.Tensor:
    d = _dims(dims)
    if out is None:
        out = torch.empty(moe_packed_bytes(d), dtype=torch.uint8, device=q_gate.device)
    rc = lib().moe_pack(ctypes.byref(d), _p(q_gate), _p(s_gate), _p(q_up), _p(s_up), _p(q_down), _p(s_down),
                        _p(g3), _p(out), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_pack")
    return out


def moe_unpack(dims, packed, stream=None):
    d = _dims(dims)
    H, I = d.hidden, d.inter
    dev = packed.device
    b = _CODE_BITS.get(d.wfmt, 4)
    qg = torch.empty((I, H * b // 8), dtype=torch.uint8, device=dev)
    qu = torch.empty_like(qg)
    qd = torch.empty((H, I * b // 8), dtype=torch.uint8, device=dev)
    if d.wfmt != MOE_W_E2M1_B16:
        sg = torch.empty(I, dtype=torch.float16, device=dev)
        su = torch.empty_like(sg)
        sd = torch.empty(H, dtype=torch.float16, device=dev)
    else:
        sg = torch.empty((I, H // 16), dtype=torch.uint8, device=dev)
        su = torch.empty_like(sg)
        sd = torch.empty((H, I // 16), dtype=torch.uint8, device=dev)
    g3 = torch.empty(4, dtype=torch.float32, device=dev)
    rc = lib().moe_unpack(ctypes.byref(d), _p(packed), _p(qg), _p(sg), _p(qu), _p(su), _p(qd), _p(sd), _p(g3),
                          _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_unpack")
    return qg, sg, qu, su, qd, sd, g3[:3]


class PackedLayer:
    """Device-resident packed weights of one layer plus the expert pointer
    table that the C ABI takes (a device array of device pointers)."""

    def __init__(self, dims, packed: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor]):
        self.dims = dims
        self.packed = packed  # uint8 [E + S][packed_bytes]
        self.router_w = router_w.contiguous()
        self.router_b = None if router_b is None else router_b.contiguous()
        pb = packed.shape[1]
        base = packed.data_ptr()
        E = dims.n_experts
        self.table = torch.tensor([base + e * pb for e in range(E)], dtype=torch.int64, device=packed.device)
        self.shared_ptr = base + E * pb if dims.has_shared else None

    @classmethod
    def from_layer(cls, layer, device="cuda", stream=None):
        """Pack a canonical synth.Layer (weights on any device) onto `device`."""
        d = layer.dims
        pb = moe_packed_bytes(d)
        n = layer.q_gate.shape[0]
        packed = torch.empty((n, pb), dtype=torch.uint8, device=device)
        for e in range(n):
            t = [getattr(layer, a)[e].to(device).contiguous() for a in
                 ("q_gate", "s_gate", "q_up", "s_up", "q_down", "s_down")]
            g3 = layer.g3[e].to(device).contiguous()
            moe_pack(d, *t, g3=g3, out=packed[e], stream=stream)
        rb = None if layer.router_b is None else layer.router_b.to(device)
        return cls(d, packed, layer.router_w.to(device), rb)

    def clone(self):
        """Same weights at new device addresses."""
        return PackedLayer(self.dims, self.packed.clone(), self.router_w.clone(),
                           None if self.router_b is None else self.router_b.clone())

    def weights(self) -> MoeWeights:
        return MoeWeights(self.table.data_ptr(), self.shared_ptr, self.router_w.data_ptr(),
                          None if self.router_b is None else self.router_b.data_ptr())


def moe_route(layer: PackedLayer, x: torch.Tensor, ws: Optional[torch.Tensor] = None, stream=None):
    d = _dims(layer.dims)
    T = x.shape[0]
    k, E = d.top_k, d.n_experts
    dev = x.device
    cap = max(1, min(E, T * k))
    out = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=dev),
               topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
               n_unique=torch.zeros(4, dtype=torch.int32, device=dev),
               uniq_ids=torch.full((cap,), -1, dtype=torch.int32, device=dev),
               uniq_off=torch.full((cap + 4,), -1, dtype=torch.int32, device=dev),
               pairs=torch.full((max(1, T * k),), -1, dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(d, T, dev)
    w = layer.weights()
    rc = lib().moe_route(ctypes.byref(d), ctypes.byref(w), _p(x), T, _p(out["topk_idx"]), _p(out["topk_w"]),
                         _p(out["n_unique"]), _p(out["uniq_ids"]), _p(out["uniq_off"]), _p(out["pairs"]),
                         _p(ws), ws.numel(), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_route")
    return out


def moe_w4a16_forward(layer: PackedLayer, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                      topk_w: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    d = _dims(layer.dims)
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, d.hidden), dtype=torch.float16, device=x.device)
    if ws is None:
        ws = workspace(d, T, x.device)
    w = layer.weights()
    rc = lib().moe_w4a16_forward(ctypes.byref(d), ctypes.byref(w), _p(x), T, _p(y), _p(topk_idx), _p(topk_w),
                                 _p(ws), ws.numel(), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w4a16_forward")
    return y


def moe_w4a16_forward_noalloc(layer: PackedLayer, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                              topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """moe_w4a16_forward without a workspace: the library's fixed per-GPU
    scratch array serves instead (the call allocates nothing on the device;
    pass `y` to allocate nothing here either)."""
    d = _dims(layer.dims)
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, d.hidden), dtype=torch.float16, device=x.device)
    w = layer.weights()
    rc = lib().moe_w4a16_forward_noalloc(ctypes.byref(d), ctypes.byref(w), _p(x), T, _p(y), _p(topk_idx),
                                         _p(topk_w), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w4a16_forward_noalloc")
    return y


def moe_w4a16_forward_profiled(layer: PackedLayer, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor, events,
                               stream=None) -> torch.Tensor:
    """moe_w4a16_forward that times its stages: `events` holds up to six raw
    hipEvent_t handles (ints, or None); events[2i] / events[2i+1] take the
    start / end of stage i (0 route, 1 gate/up, 2 down), recorded by the
    stage's first / last kernel dispatch."""
    d = _dims(layer.dims)
    T = x.shape[0]
    handles = (ctypes.c_void_p * len(events))(*events)
    w = layer.weights()
    rc = lib().moe_w4a16_forward_profiled(ctypes.byref(d), ctypes.byref(w), _p(x), T, _p(y), None, None, _p(ws),
                                          ws.numel(), _stream(stream), handles, len(events))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w4a16_forward_profiled")
    return y


class StepGraph:
    """Several layer calls captured once as one HIP graph by the library
    (moe_step_graph_create) and replayed with one launch.  Layer l reads
    xs[l] and writes ys[l] (pass ys[l] as xs[l + 1] to chain the layers);
    all layers share the workspace `ws`.  The tensors must stay alive, at the
    same addresses, for the life of the graph."""

    def __init__(self, layers, xs, ys, ws: Optional[torch.Tensor] = None):
        if not (len(layers) == len(xs) == len(ys)) or not layers:
            raise ValueError("one input and one output per layer")
        d = _dims(layers[0].dims)
        T = xs[0].shape[0]
        if ws is None:
            ws = workspace(d, T, xs[0].device)
        self._keep = (list(layers), list(xs), list(ys), ws)
        n = len(layers)
        w = (MoeWeights * n)(*[pl.weights() for pl in layers])
        xp = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
        yp = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
        h = ctypes.c_void_p()
        rc = lib().moe_step_graph_create(ctypes.byref(d), n, w, xp, T, yp, _p(ws), ws.numel(), ctypes.byref(h))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_step_graph_create")
        self._h = h

    def launch(self, stream=None):
        rc = lib().moe_step_graph_launch(self._h, _stream(stream))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_step_graph_launch")

    def close(self):
        if getattr(self, "_h", None):
            rc = lib().moe_step_graph_destroy(self._h)
            self._h = None
            if rc != MOE_OK:
                raise MoeError(rc, "moe_step_graph_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def probe_stream_read(buf: torch.Tensor, blocks: int, sink: torch.Tensor, stream=None):
    """One plain streaming read of `buf` (moe_probe_stream_read)."""
    rc = lib().moe_probe_stream_read(_p(buf), buf.numel() * buf.element_size(), _p(sink), blocks, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_probe_stream_read")


def probe_mfma(sink: torch.Tensor, blocks: int, iters: int, stream=None) -> int:
    """One pure matrix-core loop (moe_probe_mfma); returns its fp16 flops."""
    rc = lib().moe_probe_mfma(_p(sink), blocks, iters, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_probe_mfma")
    return blocks * 8 * iters * 16 * 2 * 16 * 16 * 32


# ---- tiered expert residency (include/moe_tier.h) ---------------------------
class Tier:
    """A moe_tier manager.  `host_ptrs` are the (host) addresses of the packed
    experts of every layer, layer-major; `slots` / `table` are device tensors
    (None for the bookkeeping-only dry mode); `copy_stream` a torch stream."""

    def __init__(self, dims, n_layers: int, host_ptrs, slots_per_layer: int, slots=None, table=None,
                 copy_stream=None, policy: int = MOE_TIER_LRU):
        self.dims = _dims(dims)
        self.n_layers = n_layers
        n = n_layers * self.dims.n_experts
        if len(host_ptrs) != n:
            raise ValueError("host_ptrs must hold n_layers * n_experts addresses")
        self._host = (ctypes.c_void_p * n)(*host_ptrs)
        self.slots, self.table, self.copy_stream = slots, table, copy_stream
        h = ctypes.c_void_p()
        rc = lib().moe_tier_create(ctypes.byref(self.dims), n_layers, self._host, _p(slots), slots_per_layer,
                                   _p(table), None if copy_stream is None else _stream(copy_stream), int(policy),
                                   ctypes.byref(h))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_tier_create")
        self._h = h

    def close(self):
        if self._h:
            lib().moe_tier_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _call(self, fn, layer, experts, stream):
        e = (ctypes.c_int32 * len(experts))(*[int(v) for v in experts])
        s = None if self.copy_stream is None and stream is None else _stream(stream)
        rc = fn(self._h, int(layer), e, len(experts), s)
        if rc != MOE_OK:
            raise MoeError(rc, fn.__name__)

    def use(self, layer, experts, stream=None):
        self._call(lib().moe_tier_use, layer, experts, stream)

    def prefetch(self, layer, experts, stream=None):
        self._call(lib().moe_tier_prefetch, layer, experts, stream)

    def sync(self, stream=None):
        """`stream` waits for every promotion enqueued so far."""
        rc = lib().moe_tier_sync(self._h, None if self.copy_stream is None and stream is None else _stream(stream))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_tier_sync")

    def slot(self, layer, expert) -> int:
        return int(lib().moe_tier_slot(self._h, int(layer), int(expert)))

    def stats(self) -> dict:
        st = MoeTierStats()
        rc = lib().moe_tier_stats(self._h, ctypes.byref(st))
        if rc != MOE_OK:
            raise MoeError(rc, "moe_tier_stats")
        return {f: int(getattr(st, f)) for f, _ in MoeTierStats._fields_}

    def weights(self, layer, router_w, router_b, shared_ptr) -> MoeWeights:
        """moe_weights_t of one layer that reads its experts through the table."""
        ptr = self.table.data_ptr() + layer * self.dims.n_experts * 8
        return MoeWeights(ptr, shared_ptr, router_w.data_ptr(), None if router_b is None else router_b.data_ptr())


from .dispatch import (MOE_T_BF16, MOE_T_F16, MOE_T_F32, moe_combine, moe_combine_backward, moe_dispatch,  # noqa: E402
                       moe_dispatch_backward, moe_route_backward, moe_sort, moe_sort_rows)
from .adapter import moe_adapter_backward, moe_adapter_forward  # noqa: E402
from .w4 import W4Weights, moe_w4_backward, moe_w4_few_rows, moe_w4_forward, moe_w4_pack, moe_w4_unpack  # noqa: E402
from .distill import moe_distill_backward, moe_distill_forward  # noqa: E402
