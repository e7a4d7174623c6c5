"""Python binding of libmoe.so, the GB300 (sm_103a) routed-expert MoE FFN layer.

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  The functions carry the C ABI's names (include/moe.h) and take
plain integers for device pointers and streams, so any allocator can feed
them; the `Layer` helper adds torch-tensor convenience on top (torch is used
for device memory and streams, nothing else).

There is no fallback: if libmoe.so is missing or cannot be loaded, every
call raises MoeError.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

__all__ = [
    "MoeError", "MoeDesc", "MoeWeights", "MoeRouteOut", "MODE_ROUTE", "MODE_PREFILL", "MODE_DECODE",
    "DECODE_MAX_T", "moe_create", "moe_destroy", "moe_workspace_bytes", "moe_route", "moe_route_from_logits",
    "moe_route_from_logits_noalloc", "moe_forward_prefill", "moe_forward_decode", "moe_forward_host", "moe_get_device_status",
    "moe_set_wait_limit", "moe_debug_timeout_probe", "moe_debug_inject", "moe_profile_enable", "moe_profile_read", "moe_status_string", "moe_last_error",
    "moe_abi_version", "moe_forward_smallep", "moe_forward_deferred", "moe_layers_workspace_bytes",
    "moe_forward_layers", "smallep_groups", "moe_create_ex", "moe_tiles_bytes", "moe_tiles_load", "moe_forward_tiles",
    "CREATE_HOST_TILES", "library_path", "load", "Layer", "LayerStackGraph", "StreamedStack",
    "MoeFp8Matrix", "MoeRmsnormArgs", "MoeLinearDesc", "MoeLinearWeights", "BF16", "F32", "SCALE_F32", "SCALE_E8M0",
    "moe_add_rmsnorm", "moe_rmsnorm_device_status", "moe_rmsnorm_set_wait_limit", "moe_rmsnorm_debug_timeout", "moe_linear_create", "moe_linear_destroy", "moe_linear_forward", "moe_gated_linear_forward",
    "moe_linear_device_status", "moe_linear_set_wait_limit", "moe_linear_debug_timeout", "Fp8Tensor", "RmsNorm", "Fp8Linear", "Fp8GatedLinear", "DenseFfn",
]

MODE_ROUTE, MODE_PREFILL, MODE_DECODE = 0, 1, 2
CREATE_HOST_TILES = 1
DECODE_MAX_T = 64
BF16, F32 = 0, 1
SCALE_F32, SCALE_E8M0 = 0, 1
MOE_OK = 0
DEV_BAD_EXPERT_ID, DEV_BAD_ROW, DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class MoeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "inter", "n_experts", "top_k", "n_shared", "shared_inter")]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "router_w", "router_bias", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
        "sh_gate", "sh_up", "sh_down", "sh_s_gate", "sh_s_up", "sh_s_down")]


class MoeRouteOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "logits", "topk_ids", "topk_w", "expert_offsets", "sorted_token", "inv_row", "xq", "sx", "hq", "sh")]


class MoeFp8Matrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("lds", ctypes.c_int64),
                ("scale_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoeRmsnormArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("res_type", ctypes.c_int32), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("res", ctypes.c_void_p), ("ld_res", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("res_out", ctypes.c_void_p), ("ld_res_out", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("out", MoeFp8Matrix), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class MoeLinearDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_features", "out_features", "gated", "scale_type")]


class MoeLinearWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w", "s", "w_up", "s_up")]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load libmoe.so (optionally building it first).  The environment
    variable MOE_LIBRARY, if set, names another build of the library to load."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = os.environ.get("MOE_LIBRARY") or _build.LIB
        if build_if_missing and path == _build.LIB and not _build.up_to_date():
            _build.build()
        if not os.path.exists(path):
            raise MoeError(-1, f"libmoe.so is not built ({path}); run __graft_entry__.build() first")
        try:
            lib = ctypes.CDLL(path)
        except OSError as e:
            raise MoeError(-1, f"cannot load {path}: {e}") from e
        vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        st = ctypes.c_int
        sig = {
            "moe_create": ([ctypes.POINTER(MoeDesc), ctypes.POINTER(MoeWeights), vp, ctypes.POINTER(vp)], st),
            "moe_destroy": ([vp], st),
            "moe_workspace_bytes": ([vp, i32, i32, ctypes.POINTER(sz)], st),
            "moe_route": ([vp, vp, i32, ctypes.POINTER(MoeRouteOut), vp, sz, vp], st),
            "moe_route_from_logits": ([vp, vp, i32, ctypes.POINTER(MoeRouteOut), vp, sz, vp], st),
            "moe_forward_prefill": ([vp, vp, i32, vp, ctypes.POINTER(MoeRouteOut), vp, sz, vp], st),
            "moe_forward_decode": ([vp, vp, i32, vp, ctypes.POINTER(MoeRouteOut), vp, sz, vp], st),
            "moe_forward_host": ([vp, i32, vp, i32, vp, vp, sz, vp], st),
            "moe_get_device_status": ([vp, vp, ctypes.POINTER(u32)], st),
            "moe_set_wait_limit": ([vp, u32], st),
            "moe_debug_timeout_probe": ([vp, vp], st),
            "moe_debug_inject": ([vp, u32], st),
            "moe_route_from_logits_noalloc": ([vp, vp, i32, ctypes.POINTER(MoeRouteOut), vp], st),
            "moe_forward_smallep": ([vp, i32, i32, vp, i32, vp, vp, sz, vp], st),
            "moe_create_ex": ([ctypes.POINTER(MoeDesc), ctypes.POINTER(MoeWeights), u32, vp, ctypes.POINTER(vp)], st),
            "moe_tiles_bytes": ([vp, ctypes.POINTER(sz)], st),
            "moe_tiles_load": ([vp, vp, vp], st),
            "moe_forward_tiles": ([vp, i32, vp, vp, i32, vp, vp, sz, vp], st),
            "moe_forward_deferred": ([vp, i32, vp, i32, vp, vp, vp, vp, sz, vp], st),
            "moe_layers_workspace_bytes": ([ctypes.POINTER(vp), i32, i32, i32, ctypes.POINTER(sz)], st),
            "moe_forward_layers": ([ctypes.POINTER(vp), i32, i32, vp, i32, vp, vp, sz, vp], st),
            "moe_profile_enable": ([vp, i32], st),
            "moe_profile_read": ([vp, ctypes.POINTER(ctypes.c_float), i32], st),
            "moe_add_rmsnorm": ([ctypes.POINTER(MoeRmsnormArgs), vp], st),
            "moe_rmsnorm_device_status": ([vp, ctypes.POINTER(u32)], st),
            "moe_rmsnorm_set_wait_limit": ([u32], st),
            "moe_rmsnorm_debug_timeout": ([], st),
            "moe_linear_create": ([ctypes.POINTER(MoeLinearDesc), ctypes.POINTER(MoeLinearWeights), vp,
                                   ctypes.POINTER(vp)], st),
            "moe_linear_destroy": ([vp], st),
            "moe_linear_forward": ([vp, ctypes.POINTER(MoeFp8Matrix), i32, vp, ctypes.c_int64, i32, vp], st),
            "moe_gated_linear_forward": ([vp, ctypes.POINTER(MoeFp8Matrix), i32, ctypes.POINTER(MoeFp8Matrix), vp], st),
            "moe_linear_device_status": ([vp, vp, ctypes.POINTER(u32)], st),
            "moe_linear_set_wait_limit": ([vp, u32], st),
            "moe_linear_debug_timeout": ([vp], st),
            "moe_status_string": ([st], ctypes.c_char_p),
            "moe_last_error": ([], ctypes.c_char_p),
            "moe_abi_version": ([], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(status: int):
    if status != MOE_OK:
        lib = load()
        raise MoeError(status, f"{lib.moe_status_string(status).decode()}: {lib.moe_last_error().decode()}")


def _route_out(out):
    if out is None:
        return None
    if isinstance(out, MoeRouteOut):
        return ctypes.byref(out)
    return ctypes.byref(MoeRouteOut(**{k: v for k, v in out.items() if v}))


# ---------------------------------------------------------------- ABI functions

def moe_abi_version() -> int:
    return int(load().moe_abi_version())


def moe_status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def moe_last_error() -> str:
    return load().moe_last_error().decode()


def moe_create(desc: MoeDesc, weights: MoeWeights, stream: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(load().moe_create(ctypes.byref(desc), ctypes.byref(weights), stream, ctypes.byref(h)))
    return h.value


def moe_create_ex(desc: MoeDesc, weights: MoeWeights, flags: int, stream: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(load().moe_create_ex(ctypes.byref(desc), ctypes.byref(weights), flags, stream, ctypes.byref(h)))
    return h.value


def moe_tiles_bytes(layer: int) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_tiles_bytes(layer, ctypes.byref(n)))
    return n.value


def moe_tiles_load(layer: int, slot: int, stream: int = 0) -> None:
    _check(load().moe_tiles_load(layer, slot, stream))


def moe_forward_tiles(layer: int, mode: int, slot: int, x: int, T: int, y: int, ws: int, ws_bytes: int,
                      stream: int = 0) -> None:
    _check(load().moe_forward_tiles(layer, mode, slot, x, T, y, ws, ws_bytes, stream))


def moe_destroy(layer: int) -> None:
    _check(load().moe_destroy(layer))


def moe_workspace_bytes(layer: int, T: int, mode: int) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_workspace_bytes(layer, T, mode, ctypes.byref(n)))
    return n.value


def moe_route(layer: int, x: int, T: int, out, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check(load().moe_route(layer, x, T, _route_out(out), ws, ws_bytes, stream))


def moe_route_from_logits(layer: int, logits: int, T: int, out, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check(load().moe_route_from_logits(layer, logits, T, _route_out(out), ws, ws_bytes, stream))


def moe_route_from_logits_noalloc(layer: int, logits: int, T: int, out, stream: int = 0) -> None:
    """Routing from given logits with the library's built-in scratch (no
    workspace, no allocation) -- for callers that cannot allocate device
    memory when they route.  See include/moe.h for the size limit."""
    _check(load().moe_route_from_logits_noalloc(layer, logits, T, _route_out(out), stream))


def moe_forward_prefill(layer: int, x: int, T: int, y: int, dbg, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check(load().moe_forward_prefill(layer, x, T, y, _route_out(dbg), ws, ws_bytes, stream))


def moe_forward_decode(layer: int, x: int, T: int, y: int, dbg, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check(load().moe_forward_decode(layer, x, T, y, _route_out(dbg), ws, ws_bytes, stream))


def moe_forward_host(layer: int, mode: int, x_host: int, T: int, y_host: int, ws: int, ws_bytes: int,
                     stream: int = 0) -> None:
    _check(load().moe_forward_host(layer, mode, x_host, T, y_host, ws, ws_bytes, stream))


def moe_forward_smallep(layer: int, mode: int, n_ranks: int, x: int, T: int, y: int, ws: int, ws_bytes: int,
                        stream: int = 0) -> None:
    _check(load().moe_forward_smallep(layer, mode, n_ranks, x, T, y, ws, ws_bytes, stream))


def smallep_groups(n_experts: int, n_ranks: int):
    """Expert range [lo, hi) of each SmallEP rank, as moe_forward_smallep
    splits them: rank p holds [ceil(p E / P), ceil((p + 1) E / P)); rank 0
    also holds the shared expert."""
    b = [(p * n_experts + n_ranks - 1) // n_ranks for p in range(n_ranks + 1)]
    return [(b[p], b[p + 1]) for p in range(n_ranks)]


def moe_forward_deferred(layer: int, mode: int, x: int, T: int, defer: int, y_now: int, y_next: int, ws: int,
                         ws_bytes: int, stream: int = 0) -> None:
    _check(load().moe_forward_deferred(layer, mode, x, T, defer, y_now, y_next, ws, ws_bytes, stream))


def _handles(layers):
    arr = (ctypes.c_void_p * len(layers))(*[int(h) for h in layers])
    return arr


def moe_layers_workspace_bytes(layers, T: int, mode: int) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_layers_workspace_bytes(_handles(layers), len(layers), T, mode, ctypes.byref(n)))
    return n.value


def moe_forward_layers(layers, mode: int, x: int, T: int, y: int, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check(load().moe_forward_layers(_handles(layers), len(layers), mode, x, T, y, ws, ws_bytes, stream))


def moe_get_device_status(layer: int, stream: int = 0):
    """Returns (status, flags) without raising, so callers can inspect both."""
    f = ctypes.c_uint32()
    st = load().moe_get_device_status(layer, stream, ctypes.byref(f))
    return int(st), int(f.value)


def moe_set_wait_limit(layer: int, microseconds: int) -> None:
    _check(load().moe_set_wait_limit(layer, microseconds))


def moe_debug_timeout_probe(layer: int, stream: int = 0) -> None:
    _check(load().moe_debug_timeout_probe(layer, stream))


def moe_debug_inject(layer: int, faults: int) -> None:
    """Plant the faults (DEV_BAD_EXPERT_ID | DEV_BAD_ROW) in the next routing
    or forward call's workspace; the kernels must flag them and stay in
    bounds (test hook, see include/moe.h)."""
    _check(load().moe_debug_inject(layer, faults))


PROFILE_STAGES = ("route", "quant_x", "gate_up", "down", "combine")


PROFILE_SELECT = 0x40000000


def moe_profile_enable(layer: int, enable: bool = True, stages=None) -> None:
    """Record stage events in forward calls: every stage, or only the named
    ones (e.g. stages=("gate_up",)); enable=False turns profiling off."""
    if not enable:
        code = 0
    elif stages is None:
        code = 1
    else:
        code = PROFILE_SELECT
        for name in stages:
            code |= 1 << PROFILE_STAGES.index(name)
    _check(load().moe_profile_enable(layer, code))


def moe_profile_read(layer: int):
    """Elapsed ms of each stage of the most recent forward call (dict); -1
    for a stage that is not timed."""
    buf = (ctypes.c_float * len(PROFILE_STAGES))()
    _check(load().moe_profile_read(layer, buf, len(PROFILE_STAGES)))
    return dict(zip(PROFILE_STAGES, [float(v) for v in buf]))


def moe_add_rmsnorm(args: MoeRmsnormArgs, stream: int = 0) -> None:
    _check(load().moe_add_rmsnorm(ctypes.byref(args), stream))


def moe_rmsnorm_device_status(stream: int = 0):
    """Returns (status, flags) without raising, so callers can inspect both."""
    f = ctypes.c_uint32()
    st = load().moe_rmsnorm_device_status(stream, ctypes.byref(f))
    return int(st), int(f.value)


def moe_rmsnorm_set_wait_limit(microseconds: int) -> None:
    _check(load().moe_rmsnorm_set_wait_limit(microseconds))


def moe_rmsnorm_debug_timeout() -> None:
    """In the next norm of many rows that copies them to shared memory first, the wait for one row expires."""
    _check(load().moe_rmsnorm_debug_timeout())


def moe_linear_create(desc: MoeLinearDesc, weights: MoeLinearWeights, stream: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(load().moe_linear_create(ctypes.byref(desc), ctypes.byref(weights), stream, ctypes.byref(h)))
    return h.value


def moe_linear_destroy(linear: int) -> None:
    _check(load().moe_linear_destroy(linear))


def moe_linear_forward(linear: int, a: MoeFp8Matrix, rows: int, y: int, ldy: int, y_type: int,
                       stream: int = 0) -> None:
    _check(load().moe_linear_forward(linear, ctypes.byref(a), rows, y, ldy, y_type, stream))


def moe_gated_linear_forward(linear: int, a: MoeFp8Matrix, rows: int, h: MoeFp8Matrix, stream: int = 0) -> None:
    _check(load().moe_gated_linear_forward(linear, ctypes.byref(a), rows, ctypes.byref(h), stream))


def moe_linear_device_status(linear: int, stream: int = 0):
    """Returns (status, flags) without raising, so callers can inspect both."""
    f = ctypes.c_uint32()
    st = load().moe_linear_device_status(linear, stream, ctypes.byref(f))
    return int(st), int(f.value)


def moe_linear_set_wait_limit(linear: int, microseconds: int) -> None:
    _check(load().moe_linear_set_wait_limit(linear, microseconds))


def moe_linear_debug_timeout(linear: int) -> None:
    """In the next forward call of this projection the wait for the last products of one tile expires."""
    _check(load().moe_linear_debug_timeout(linear))


# ---------------------------------------------------------------- torch convenience

class Layer:
    """A layer built from torch CUDA tensors (checkpoint layout, see moe.h).

    weights: dict with router_w, router_b (or None), w_gate, w_up, w_down,
    s_gate, s_up, s_down and, with a shared expert, sh_* of the same layout.
    The library copies the weights; the tensors may be freed afterwards.
    """

    def __init__(self, hidden, inter, n_experts, top_k, weights: dict, n_shared: int = 1, stream=None,
                 host_tiles: bool = False):
        import torch
        self.desc = MoeDesc(hidden, inter, n_experts, top_k, n_shared, inter if n_shared else 0)
        p = lambda n: (weights[n].data_ptr() if weights.get(n) is not None else None)
        self.weights = MoeWeights(
            p("router_w"), p("router_b"), p("w_gate"), p("w_up"), p("w_down"), p("s_gate"), p("s_up"), p("s_down"),
            p("sh_gate"), p("sh_up"), p("sh_down"), p("sh_s_gate"), p("sh_s_up"), p("sh_s_down"))
        self.stream = stream if stream is not None else torch.cuda.current_stream().cuda_stream
        self.handle = moe_create_ex(self.desc, self.weights, CREATE_HOST_TILES if host_tiles else 0, self.stream)
        self._ws = {}

    def workspace(self, T: int, mode: int):
        import torch
        need = moe_workspace_bytes(self.handle, T, mode)
        if mode == MODE_PREFILL or mode == MODE_DECODE:
            need += 4 * T * self.desc.hidden + 1024     # room for moe_forward_host's device copies
        cur = self._ws.get("buf")
        if cur is None or cur.numel() < need:
            self._ws["buf"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        buf = self._ws["buf"]
        return buf.data_ptr(), buf.numel()

    def close(self):
        if self.handle:
            moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LayerStackGraph:
    """A stack of layers (handles) run as one moe_forward_layers call,
    captured once into a CUDA graph and replayed: the whole decode step is a
    single graph launch.  x and y are torch CUDA bf16-bits tensors [T][H]
    owned by the caller; replay() runs the stack on the current contents of
    x and leaves the result in y."""

    def __init__(self, handles, mode: int, x, y, warmup: int = 1):
        import torch
        self.handles = list(handles)
        self.mode = mode
        self.x, self.y = x, y
        T = x.shape[0]
        need = moe_layers_workspace_bytes(self.handles, T, mode)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
        self.stream = torch.cuda.Stream(device=x.device)
        run = lambda: moe_forward_layers(self.handles, mode, x.data_ptr(), T, y.data_ptr(), self.ws.data_ptr(),
                                         self.ws.numel(), self.stream.cuda_stream)
        with torch.cuda.stream(self.stream):
            for _ in range(warmup):           # one-time kernel attributes are set outside the capture
                run()
        self.stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            run()

    def replay(self):
        """Launch the captured stack on the current torch stream."""
        self.graph.replay()


class StreamedStack:
    """A stack of host-tile layers (moe_create_ex with CREATE_HOST_TILES) run
    through a two-slot device ring: while layer l computes from slot l % 2,
    a copy stream loads layer l + 1's tiles into the other slot (ordered by
    events: a slot is reloaded only after the layer that read it finished).
    x and y: torch CUDA [T][H] bf16-bits tensors; run() computes on the
    current torch stream and returns when the work is enqueued."""

    def __init__(self, layers, mode: int, x, y):
        import torch
        self.layers = list(layers)
        self.mode, self.x, self.y = mode, x, y
        T = x.shape[0]
        slot_bytes = max(moe_tiles_bytes(ly.handle) for ly in self.layers)
        self.slots = [torch.empty(slot_bytes, dtype=torch.uint8, device=x.device) for _ in range(2)]
        self.acts = [torch.empty_like(x) for _ in range(2)]
        need = max(moe_workspace_bytes(ly.handle, T, mode) for ly in self.layers)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
        self.copy = torch.cuda.Stream(device=x.device)
        self.loaded = [torch.cuda.Event() for _ in range(2)]
        self.done = [torch.cuda.Event() for _ in range(2)]

    def run(self):
        import torch
        comp = torch.cuda.current_stream()
        n, T = len(self.layers), self.x.shape[0]

        def load_into(l):
            s = l % 2
            self.copy.wait_event(self.done[s]) if l >= 2 else self.copy.wait_stream(comp)
            moe_tiles_load(self.layers[l].handle, self.slots[s].data_ptr(), self.copy.cuda_stream)
            self.loaded[s].record(self.copy)

        load_into(0)
        for l in range(n):
            if l + 1 < n:
                load_into(l + 1)
            s = l % 2
            comp.wait_event(self.loaded[s])
            src = self.x if l == 0 else self.acts[(l - 1) % 2]
            dst = self.y if l == n - 1 else self.acts[l % 2]
            moe_forward_tiles(self.layers[l].handle, self.mode, self.slots[s].data_ptr(), src.data_ptr(), T,
                              dst.data_ptr(), self.ws.data_ptr(), self.ws.numel(), comp.cuda_stream)
            self.done[s].record(comp)


# ---------------------------------------------------------------- dense operators (torch convenience)

MOE_ERR_INVALID_ARG = 1
_SCALES = {"f32": SCALE_F32, "e8m0": SCALE_E8M0}


def _bad(message: str):
    raise MoeError(MOE_ERR_INVALID_ARG, message)


_current = None          # torch's functions for the current device and a device's current stream, looked up once


def _stream(dev: int) -> int:
    """The current torch stream's handle on device `dev`, which has to be the
    current device.  torch.cuda.current_stream() builds a Python object, which
    takes longer than a small operator's launch; the raw handle does not."""
    global _current
    if _current is None:
        import torch
        torch.cuda.init()
        _current = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                    getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream))
    if dev != _current[0]():
        _bad(f"the tensors are on device {dev}, which is not the current one")
    return _current[1](dev)


def _dtypes():
    import torch
    return {torch.bfloat16: BF16, torch.float32: F32}


def _rows_of(t, rows: int, cols: int, dev: int, what: str) -> int:
    """Row stride of a [rows][cols] tensor with contiguous rows on device `dev`."""
    if t.shape != (rows, cols):
        _bad(f"{what} must be [{rows}][{cols}], not {list(t.shape)}")
    if t.get_device() != dev:
        _bad(f"{what} must be on CUDA device {dev}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        _bad(f"{what} must have contiguous rows")
    return ld if rows > 1 or ld >= cols else cols


class Fp8Tensor:
    """E4M3 activations with 1x128 scales: value = q * s[column // 128].

    q: float8_e4m3fn [rows][cols]; s: [ceil(cols / 128)][rows], float32
    (scale="f32") or float8_e8m0fnu (scale="e8m0").  Rows of both lie on
    16-byte strides.  matrix is the C ABI's view of them."""

    def __init__(self, rows: int, cols: int, scale: str = "f32", device=None):
        import torch
        if scale not in _SCALES:
            _bad(f"scale must be one of {sorted(_SCALES)}, not {scale!r}")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        st = torch.float32 if scale == "f32" else torch.float8_e8m0fnu
        q = torch.empty(rows, _up(cols, 16), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)[:, :cols]
        s = torch.empty(_up(cols, 128) // 128, _up(rows, 16), dtype=torch.uint8 if scale == "e8m0" else st, device=device)
        self._bind(q, s.view(st)[:, :rows], scale)

    def _bind(self, q, s, scale):
        self.rows, self.cols, self.scale, self.q, self.s = q.shape[0], q.shape[1], scale, q, s
        self.device, self._dev = q.device, q.get_device()
        self.matrix = MoeFp8Matrix(q.data_ptr(), s.data_ptr(), q.stride(0), s.stride(0), _SCALES[scale], 0)
        self._ref = ctypes.byref(self.matrix)
        self._packed = (q.data_ptr(), s.data_ptr(), q.stride(0), s.stride(0), _SCALES[scale])

    @classmethod
    def from_parts(cls, q, s):
        """Wrap codes and scales that exist already; an array whose rows do
        not lie on 16-byte strides is copied."""
        import torch
        if q.dim() != 2 or q.dtype is not torch.float8_e4m3fn or not q.is_cuda:
            _bad("q must be a two-dimensional float8_e4m3fn CUDA tensor")
        scale = {torch.float32: "f32", torch.float8_e8m0fnu: "e8m0"}.get(s.dtype)
        rows, cols = q.shape
        if scale is None or s.device != q.device or list(s.shape) != [_up(cols, 128) // 128, rows]:
            _bad(f"s must be float32 or float8_e8m0fnu [{_up(cols, 128) // 128}][{rows}] beside q")
        t = cls.__new__(cls)
        t._bind(_on_strides(q), _on_strides(s), scale)
        return t

    def first(self, rows: int):
        """The first rows as an Fp8Tensor over the same storage."""
        t = type(self).__new__(type(self))
        t._bind(self.q[:rows], self.s[:, :rows], self.scale)
        return t

    def dequantise(self):
        """The values the codes stand for, fp32."""
        return self.q.float() * self.s.float().t().repeat_interleave(128, 1)[:, :self.cols]


def _up(n: int, to: int) -> int:
    return (n + to - 1) // to * to


def _on_strides(t):
    """t itself if it has contiguous rows on 16-byte strides, else a copy that has."""
    import torch
    n, es = t.shape[1], t.element_size()
    if t.data_ptr() % 16 == 0 and t.stride(1) == 1 and t.stride(0) >= n and t.stride(0) * es % 16 == 0:
        return t
    bits = torch.uint8 if es == 1 else t.dtype
    wide = torch.zeros(t.shape[0], _up(n, 16), dtype=bits, device=t.device)
    wide[:, :n] = t.view(bits)
    return wide.view(t.dtype)[:, :n]


# MoeRmsnormArgs as one packed block: filling the ctypes structure field by field takes longer than the launch
_RMSNORM_ARGS = struct.Struct("@iiiiPqPqPPqPqPPqqiifi")
assert _RMSNORM_ARGS.size == ctypes.sizeof(MoeRmsnormArgs)
_NO_OUT = (0, 0, 0, 0, 0)


class RmsNorm:
    """v = x + residual; n = v * rsqrt(mean(v^2) + eps) * weight.

    Calling it writes whichever outputs are given: res_out (v, in the
    residual's type; may be the residual itself), y (n, in x's type) and out
    (n quantised, an Fp8Tensor)."""

    def __init__(self, weight, eps: float = 1e-6):
        import torch
        if weight.dim() != 1 or not weight.is_cuda:
            _bad("weight must be a one-dimensional CUDA tensor")
        self.weight = weight.to(torch.float32).contiguous()
        self.eps, self.cols = float(eps), weight.shape[0]
        self._w, self._dev, self._types = self.weight.data_ptr(), weight.get_device(), _dtypes()
        self._call = load()["moe_add_rmsnorm"]          # a prototype of its own, which takes the packed block
        self._call.argtypes, self._call.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int

    def __call__(self, x, residual=None, out=None, res_out=None, y=None):
        cols, dev, rows = self.cols, self._dev, x.shape[0]
        xt = rt = self._types.get(x.dtype)
        if xt is None:
            _bad(f"x must be bfloat16 or float32, not {x.dtype}")
        ldx = _rows_of(x, rows, cols, dev, "x")
        r = ldr = ro = ldro = yp = ldy = 0
        if residual is not None:
            rt = self._types.get(residual.dtype)
            if rt is None:
                _bad(f"residual must be bfloat16 or float32, not {residual.dtype}")
            r, ldr = residual.data_ptr(), _rows_of(residual, rows, cols, dev, "residual")
        if res_out is not None:
            if residual is None or res_out.dtype is not residual.dtype:
                _bad("res_out needs a residual of its type")
            ro, ldro = res_out.data_ptr(), _rows_of(res_out, rows, cols, dev, "res_out")
        if y is not None:
            if y.dtype is not x.dtype:
                _bad("y must have x's type")
            yp, ldy = y.data_ptr(), _rows_of(y, rows, cols, dev, "y")
        if out is not None and (out.rows != rows or out.cols != cols or out._dev != dev):
            _bad(f"out must be [{rows}][{cols}] on x's device")
        st = self._call(_RMSNORM_ARGS.pack(rows, cols, xt, rt, x.data_ptr(), ldx, r, ldr, self._w, ro, ldro, yp, ldy,
                                           *(_NO_OUT if out is None else out._packed), 0, self.eps, 0), _stream(dev))
        if st != MOE_OK:
            _check(st)


class _Weights:
    """Handle of one projection's weights in the library's layout."""
    gated = False

    def _create(self, mats):
        import torch
        w = mats[0][0]
        for q, s in mats:
            if q.dim() != 2 or q.dtype is not torch.float8_e4m3fn or q.shape != w.shape or not q.is_cuda:
                _bad("weights must be float8_e4m3fn [out][in] CUDA tensors of one shape")
            if s.dtype not in (torch.float32, torch.float8_e8m0fnu) or s.dtype is not mats[0][1].dtype or \
                    list(s.shape) != [(w.shape[0] + 127) // 128, (w.shape[1] + 127) // 128] or s.device != w.device:
                _bad("scales must be float32 or float8_e8m0fnu, one per 128 x 128 block")
        keep = [t.contiguous() for m in mats for t in m]
        self.out_features, self.in_features = w.shape
        self.scale = "f32" if mats[0][1].dtype is torch.float32 else "e8m0"
        self.device, self._dev, self._types = w.device, w.get_device(), _dtypes()
        self.handle = None
        self.handle = moe_linear_create(MoeLinearDesc(self.in_features, self.out_features, int(self.gated), _SCALES[self.scale]),
                                        MoeLinearWeights(*[t.data_ptr() for t in keep]), _stream(self._dev))
        lib = load()
        self._call = lib.moe_gated_linear_forward if self.gated else lib.moe_linear_forward

    def _check_a(self, a):
        if a.cols != self.in_features or a.scale != self.scale or a._dev != self._dev:
            _bad(f"a must be [rows][{self.in_features}] with {self.scale} scales on the weights' device")

    def device_status(self):
        return moe_linear_device_status(self.handle, _stream(self._dev))

    def close(self):
        if getattr(self, "handle", None):
            moe_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Fp8Linear(_Weights):
    """y = a W^T with block-scaled E4M3 on both sides.  w: float8_e4m3fn
    [out][in]; s: one scale per 128 x 128 block, float32 or float8_e8m0fnu.
    The library keeps its own copy."""

    def __init__(self, w, s):
        self._create([(w, s)])

    def __call__(self, a: Fp8Tensor, y):
        self._check_a(a)
        ldy = _rows_of(y, a.rows, self.out_features, self._dev, "y")
        yt = self._types.get(y.dtype)
        if yt is None:
            _bad(f"y must be bfloat16 or float32, not {y.dtype}")
        st = self._call(self.handle, a._ref, a.rows, y.data_ptr(), ldy, yt, _stream(self._dev))
        if st != MOE_OK:
            _check(st)
        return y


class Fp8GatedLinear(_Weights):
    """h = SiLU(a Wg^T) * (a Wu^T), written as an Fp8Tensor."""
    gated = True

    def __init__(self, w_gate, s_gate, w_up, s_up):
        self._create([(w_gate, s_gate), (w_up, s_up)])

    def __call__(self, a: Fp8Tensor, h: Fp8Tensor):
        self._check_a(a)
        if h.rows != a.rows or h.cols != self.out_features or h.scale != self.scale or h._dev != self._dev:
            _bad(f"h must be [{a.rows}][{self.out_features}] with {self.scale} scales on the weights' device")
        st = self._call(self.handle, a._ref, a.rows, h._ref, _stream(self._dev))
        if st != MOE_OK:
            _check(st)
        return h


class DenseFfn:
    """The dense FFN half of a pre-norm block:

        residual += x;  y = down(SiLU(gate(n)) * up(n)),  n = norm(residual)

    The residual is updated in place; the caller adds y to it with the next
    norm.  The intermediate E4M3 buffers are kept between calls, so calls of
    one object belong on one stream at a time.  They are made per power of two
    of rows and never freed while the object lives: a captured graph may go on
    using them whatever sizes are called in between.  Every stream that a call
    ran on is recorded with torch's allocator, so that dropping the object while
    its kernels are queued is safe (a graph needs the object as long as it is replayed)."""

    def __init__(self, norm: RmsNorm, gate_up: Fp8GatedLinear, down: Fp8Linear):
        if gate_up.in_features != norm.cols or down.in_features != gate_up.out_features or gate_up.scale != down.scale:
            _bad("norm, gate_up and down do not fit together")
        self.norm, self.gate_up, self.down = norm, gate_up, down
        self._store, self._views, self._streams = {}, {}, {}

    def buffers(self, rows: int):
        got = self._views.get(rows)
        if got is None:
            cap = 1 << max(rows - 1, 0).bit_length()
            if cap not in self._store:
                self._store[cap] = [Fp8Tensor(cap, n, self.gate_up.scale, self.gate_up.device)
                                    for n in (self.norm.cols, self.gate_up.out_features)]
                self._streams.clear()
            got = self._views[rows] = [t.first(rows) for t in self._store[cap]]
        return got

    def _record_stream(self, handle: int):
        """The current stream, seen for the first time (or since the last buffers were made), uses all of them."""
        import torch
        stream = torch.cuda.current_stream(self.down._dev)
        for pair in self._store.values():
            for t in pair:
                t.q.record_stream(stream)
                t.s.record_stream(stream)
        self._streams[handle] = True

    def __call__(self, x, residual, y):
        rows, dev = x.shape[0], self.down._dev
        # the norm refuses x and residual before it starts; y has to be refused before the residual is changed, too
        if residual is None:
            _bad("residual is None")
        if y.dtype not in self.down._types:
            _bad(f"y must be bfloat16 or float32, not {y.dtype}")
        if _rows_of(y, rows, self.down.out_features, dev, "y") < self.down.out_features:
            _bad("y's rows overlap")
        a, h = self.buffers(rows)
        stream = _stream(dev)
        if stream not in self._streams:
            self._record_stream(stream)
        self.norm(x, residual, out=a, res_out=residual)
        self.gate_up(a, h)
        return self.down(h, y)
