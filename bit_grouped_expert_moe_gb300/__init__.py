"""Python binding of the GB300 MoE-layer library (libbgmoe.so).

Argument marshalling only: torch tensors become device pointers and the
current CUDA stream is passed through; every step of the layer runs in the
library's CUDA kernels. There is no fallback: if the library is not built,
importing the entry points raises.

Entry points mirror the C ABI in include/moe.h (workspace_bytes, max_tiles,
route_blocks, route, forward, forward_residual, forward_timed, route_noalloc,
status_read, status_string, test_route_stall, test_decode_stall) and
include/attention.h (attn_workspace_bytes, attn_decode, attn_decode_timed) and
include/gdn.h (gdn_scan, gdn_scan_timed) and include/kv8.h (kv8_write,
kv8_read, kv8_workspace_bytes, kv8_attn, kv8_attn_test_stall).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbgmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE = 0, 1, 2
MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA, MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_RANGE, MOE_ERR_BOUNDS = 3, 4, 5, 6, 7
PATH_AUTO, PATH_GEMV, PATH_TENSOR_CORE, PATH_FUSED_DECODE = 0, 1, 2, 3

P = ctypes.c_void_p


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "I_shared", "E", "top_k", "group_size", "block_m")]


class AttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "D", "L_max")]


class GdnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "Hqk", "Hv", "Dk", "Dv")]


class Kv8Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "Hq", "Hkv", "D", "L_max", "block", "format", "q_stride",
                                              "kv_stride")]


class Kv8CacheC(ctypes.Structure):
    _fields_ = [(n, P) for n in ("k_codes", "v_codes", "k_scales", "v_scales")]


class QMat(ctypes.Structure):
    _fields_ = [("codes", P), ("scales", P), ("biases", P)]


class ExpertsC(ctypes.Structure):
    _fields_ = [("gate_up", QMat), ("down", QMat)]


ROUTE_FIELDS = ("ids", "weights", "gate", "counts", "offsets", "sorted", "inv",
                "tile_expert", "tile_row0", "tile_rows", "num_tiles", "status")


class RouteOutC(ctypes.Structure):
    _fields_ = [(n, P) for n in ROUTE_FIELDS]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status}){': ' + detail if detail else ''}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with bit_grouped_expert_moe_gb300._build.build()")
        L = ctypes.CDLL(LIB_PATH)
        i32, sz = ctypes.c_int32, ctypes.c_size_t
        L.moe_abi_version.restype = i32
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [i32]
        L.moe_last_error_detail.restype = ctypes.c_char_p
        sp = ctypes.POINTER(Shape)
        L.moe_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
        L.moe_max_tiles.argtypes = [sp, ctypes.POINTER(i32)]
        L.moe_route_blocks.argtypes = [sp, ctypes.POINTER(i32)]
        L.moe_route.argtypes = [sp, P, P, P, P, ctypes.POINTER(RouteOutC), P, sz, P]
        L.moe_forward.argtypes = [sp, P, P, P, ctypes.POINTER(ExpertsC), ctypes.POINTER(ExpertsC), P, P,
                                  ctypes.POINTER(RouteOutC), P, sz, P]
        L.moe_forward_residual.argtypes = [sp, P, P, ctypes.c_float, P, P, ctypes.POINTER(ExpertsC),
                                           ctypes.POINTER(ExpertsC), P, P, P, ctypes.POINTER(RouteOutC), P, sz, P]
        L.moe_forward_timed.argtypes = [sp, P, P, P, ctypes.POINTER(ExpertsC), ctypes.POINTER(ExpertsC), P, P,
                                        ctypes.POINTER(RouteOutC), P, sz, ctypes.POINTER(P), i32, P]
        L.moe_route_noalloc.argtypes = [sp, P, P, P, P, ctypes.POINTER(RouteOutC), P]
        L.moe_route_noalloc.restype = i32
        L.moe_status_read.argtypes = [P, P, ctypes.POINTER(i32)]
        L.moe_test_route_stall.argtypes = [sp, P, P, P, P, ctypes.POINTER(RouteOutC), P, sz, i32, ctypes.c_int64, P]
        L.moe_test_decode_stall.argtypes = [sp, P, P, P, ctypes.POINTER(ExpertsC), ctypes.POINTER(ExpertsC), P, P,
                                            ctypes.POINTER(RouteOutC), P, sz, i32, ctypes.c_int64, P]
        ap = ctypes.POINTER(AttnShape)
        L.moe_attn_workspace_bytes.argtypes = [ap, ctypes.POINTER(sz)]
        L.moe_attn_decode.argtypes = [ap, P, P, P, P, ctypes.c_float, P, P, sz, P]
        L.moe_attn_decode_timed.argtypes = [ap, P, P, P, P, ctypes.c_float, P, P, sz, ctypes.POINTER(P), P]
        L.moe_attn_test_stall.argtypes = [ap, P, P, P, P, ctypes.c_float, P, P, sz, i32, ctypes.c_int64, P]
        for f in ("moe_attn_workspace_bytes", "moe_attn_decode", "moe_attn_decode_timed", "moe_attn_test_stall"):
            getattr(L, f).restype = i32
        gp = ctypes.POINTER(GdnShape)
        L.moe_gdn_scan.argtypes = [gp, P, P, P, P, P, P, P, P, P, P, P]
        L.moe_gdn_scan_timed.argtypes = [gp, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(P), P]
        L.moe_gdn_scan.restype = i32
        L.moe_gdn_scan_timed.restype = i32
        kp, cp = ctypes.POINTER(Kv8Shape), ctypes.POINTER(Kv8CacheC)
        L.moe_kv8_write.argtypes = [kp, P, P, P, P, cp, P, P]
        L.moe_kv8_read.argtypes = [kp, cp, P, P, P, P, P, P]
        L.moe_kv8_workspace_bytes.argtypes = [kp, ctypes.POINTER(sz)]
        L.moe_kv8_attn.argtypes = [kp, P, cp, P, P, ctypes.c_float, P, P, sz, P]
        L.moe_kv8_attn_test_stall.argtypes = [kp, P, cp, P, P, ctypes.c_float, P, P, sz, i32, ctypes.c_int64, P]
        for f in ("moe_kv8_write", "moe_kv8_read", "moe_kv8_workspace_bytes", "moe_kv8_attn",
                  "moe_kv8_attn_test_stall"):
            getattr(L, f).restype = i32
        for f in ("moe_workspace_bytes", "moe_max_tiles", "moe_route_blocks", "moe_route", "moe_forward",
                  "moe_forward_timed", "moe_forward_residual",
                  "moe_status_read", "moe_test_route_stall", "moe_test_decode_stall"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().moe_status_string(int(s)).decode()


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where, lib().moe_last_error_detail().decode())


def make_shape(T, H, I, E=256, top_k=8, shared=True, block_m=16, group_size=64) -> Shape:
    return Shape(T, H, I, I if shared else 0, E, top_k, group_size, block_m)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def workspace_bytes(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_workspace_bytes")
    return n.value


def max_tiles(shape: Shape) -> int:
    n = ctypes.c_int32()
    _check(lib().moe_max_tiles(ctypes.byref(shape), ctypes.byref(n)), "moe_max_tiles")
    return n.value


def route_blocks(shape: Shape) -> int:
    n = ctypes.c_int32()
    _check(lib().moe_route_blocks(ctypes.byref(shape), ctypes.byref(n)), "moe_route_blocks")
    return n.value


def alloc_route_out(shape: Shape, device) -> dict:
    """Device tensors for every routing output of `shape`."""
    T, K, E = shape.T, shape.top_k, shape.E
    A = T * K
    mt = max(1, max_tiles(shape))
    i32 = dict(dtype=torch.int32, device=device)
    return dict(ids=torch.empty(max(A, 1), **i32), weights=torch.empty(max(A, 1), dtype=torch.float32, device=device),
                gate=torch.empty(max(T, 1), dtype=torch.float32, device=device), counts=torch.empty(E + 1, **i32),
                offsets=torch.empty(E + 2, **i32), sorted=torch.empty(max(A, 1), **i32), inv=torch.empty(max(A, 1), **i32),
                tile_expert=torch.empty(mt, **i32), tile_row0=torch.empty(mt, **i32), tile_rows=torch.empty(mt, **i32),
                num_tiles=torch.zeros(1, **i32), status=torch.zeros(1, **i32))


def alloc_workspace(shape: Shape, device) -> torch.Tensor:
    """A workspace buffer of moe_workspace_bytes() bytes (torch allocations are
    at least 256-byte aligned)."""
    return torch.empty(max(workspace_bytes(shape), 256), dtype=torch.uint8, device=device)


def _route_c(out: dict) -> RouteOutC:
    return RouteOutC(*[_ptr(out.get(n)) for n in ROUTE_FIELDS])


def _experts_c(ex) -> ExpertsC | None:
    """ex = ((gu_codes, gu_scales, gu_biases), (dn_codes, dn_scales, dn_biases))."""
    if ex is None:
        return None
    (gc, gs, gb), (dc, ds, db) = ex
    return ExpertsC(QMat(_ptr(gc), _ptr(gs), _ptr(gb)), QMat(_ptr(dc), _ptr(ds), _ptr(db)))


def route(shape, x, w_router, router_bias, w_shared_gate, out: dict, workspace, stream=None):
    r = _route_c(out)
    _check(lib().moe_route(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(router_bias), _ptr(w_shared_gate),
                           ctypes.byref(r), _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(stream)), "moe_route")


def route_noalloc(shape, x, w_router, router_bias, w_shared_gate, out: dict, stream=None):
    """moe_route without a workspace (the library's own static device
    scratch; see include/moe.h for the size limit and the sharing rules)."""
    r = _route_c(out)
    _check(lib().moe_route_noalloc(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(router_bias),
                                   _ptr(w_shared_gate), ctypes.byref(r), _stream(stream)), "moe_route_noalloc")


def forward(shape, x, w_router, router_bias, experts, shared, w_shared_gate, y, workspace, route_out=None,
            stream=None):
    ec = _experts_c(experts)
    sc = _experts_c(shared)
    r = _route_c(route_out) if route_out is not None else None
    _check(lib().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(router_bias), ctypes.byref(ec),
                             ctypes.byref(sc) if sc is not None else None, _ptr(w_shared_gate), _ptr(y),
                             ctypes.byref(r) if r is not None else None, _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)), "moe_forward")


def forward_residual(shape, r, w_router, router_bias, experts, shared, w_shared_gate, y, r_next, workspace,
                     norm_weight=None, norm_eps=1e-6, route_out=None, stream=None):
    """moe_forward_residual: one pre-norm MoE block. The layer runs on
    x = RMSNorm(r) (gain norm_weight, or 1), y is its output and
    r_next = bf16(r + y) the next layer's residual row (bf16 [T, H],
    distinct from r). Fused decode shapes only."""
    ec = _experts_c(experts)
    sc = _experts_c(shared)
    rc = _route_c(route_out) if route_out is not None else None
    _check(lib().moe_forward_residual(ctypes.byref(shape), _ptr(r), _ptr(norm_weight), float(norm_eps),
                                      _ptr(w_router), _ptr(router_bias), ctypes.byref(ec),
                                      ctypes.byref(sc) if sc is not None else None, _ptr(w_shared_gate), _ptr(y),
                                      _ptr(r_next), ctypes.byref(rc) if rc is not None else None, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_forward_residual")


def forward_timed(shape, x, w_router, router_bias, experts, shared, w_shared_gate, y, workspace, events=None,
                  route_out=None, path=PATH_AUTO, stream=None):
    """forward() with a chosen expert path (PATH_AUTO, PATH_GEMV,
    PATH_TENSOR_CORE) that records six caller-created CUDA events (raw
    cudaEvent_t handles, e.g. torch.cuda.Event(enable_timing=True).cuda_event
    after one record()) around its kernels when `events` is given."""
    ec = _experts_c(experts)
    sc = _experts_c(shared)
    r = _route_c(route_out) if route_out is not None else None
    ev = (P * 6)(*events) if events is not None else None
    _check(lib().moe_forward_timed(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(router_bias), ctypes.byref(ec),
                                   ctypes.byref(sc) if sc is not None else None, _ptr(w_shared_gate), _ptr(y),
                                   ctypes.byref(r) if r is not None else None, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), ev, int(path), _stream(stream)),
           "moe_forward_timed")


def test_decode_stall(shape, x, w_router, router_bias, experts, shared, w_shared_gate, y, workspace, route_out: dict,
                      stalled_block: int, timeout_ns: int, stream=None):
    """moe_test_decode_stall: the fused decode path with one block that never
    publishes the h of its gate/up items, and a short device timeout."""
    ec = _experts_c(experts)
    sc = _experts_c(shared)
    r = _route_c(route_out)
    _check(lib().moe_test_decode_stall(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(router_bias),
                                       ctypes.byref(ec), ctypes.byref(sc) if sc is not None else None,
                                       _ptr(w_shared_gate), _ptr(y), ctypes.byref(r), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), stalled_block, timeout_ns,
                                       _stream(stream)), "moe_test_decode_stall")


def status_read(status: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32()
    _check(lib().moe_status_read(_ptr(status), _stream(stream), ctypes.byref(v)), "moe_status_read")
    return v.value


def test_route_stall(shape, x, w_router, router_bias, w_shared_gate, out: dict, workspace, stalled_block: int,
                     timeout_ns: int, stream=None):
    r = _route_c(out)
    _check(lib().moe_test_route_stall(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(router_bias),
                                      _ptr(w_shared_gate), ctypes.byref(r), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), stalled_block, timeout_ns,
                                      _stream(stream)), "moe_test_route_stall")


# ----------------------------------------------------- decode attention ---

def attn_shape(B, Hq, Hkv, D, L_max) -> AttnShape:
    return AttnShape(B, Hq, Hkv, D, L_max)


def attn_workspace_bytes(shape: AttnShape) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_attn_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_attn_workspace_bytes")
    return n.value


def attn_alloc_workspace(shape: AttnShape, device) -> torch.Tensor:
    return torch.empty(max(attn_workspace_bytes(shape), 256), dtype=torch.uint8, device=device)


def attn_decode(shape, q, k_cache, v_cache, lens, o, workspace, scale=None, stream=None):
    """moe_attn_decode: q bf16 [B, Hq, D], caches bf16 [B, Hkv, L_max, D],
    lens int32 [B], o fp32 [B, Hq, D] (all on the device). The workspace's
    first int32 is the call's device status word."""
    s = 1.0 / (shape.D ** 0.5) if scale is None else float(scale)
    _check(lib().moe_attn_decode(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lens), s,
                                 _ptr(o), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "moe_attn_decode")


def attn_test_stall(shape, q, k_cache, v_cache, lens, o, workspace, stalled_block: int, timeout_ns: int,
                    scale=None, stream=None):
    """moe_attn_test_stall: attn_decode with one grid block whose producer
    issues no cache loads and a short device timeout (test only)."""
    s = 1.0 / (shape.D ** 0.5) if scale is None else float(scale)
    _check(lib().moe_attn_test_stall(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lens), s,
                                     _ptr(o), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     int(stalled_block), int(timeout_ns), _stream(stream)), "moe_attn_test_stall")


def attn_decode_timed(shape, q, k_cache, v_cache, lens, o, workspace, events, scale=None, stream=None):
    """attn_decode recording three caller-created CUDA events (raw handles)
    before the block kernel, between it and the merge kernel, and after."""
    s = 1.0 / (shape.D ** 0.5) if scale is None else float(scale)
    ev = (P * 3)(*events)
    _check(lib().moe_attn_decode_timed(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lens), s,
                                       _ptr(o), _ptr(workspace), workspace.numel() * workspace.element_size(), ev,
                                       _stream(stream)), "moe_attn_decode_timed")


# ------------------------------------------------------- Gated DeltaNet ---

def gdn_shape(B, T, Hqk, Hv, Dk=128, Dv=128) -> GdnShape:
    return GdnShape(B, T, Hqk, Hv, Dk, Dv)


def gdn_scan(shape, q, k, v, gate, beta, offsets, state_in, state_out, o, status=None, stream=None):
    """moe_gdn_scan: q, k bf16 [T, Hqk, Dk]; v bf16 [T, Hv, Dv]; gate, beta
    fp32 [T, Hv]; offsets int32 [B+1]; states fp32 [B, Hv, Dv, Dk] (state_out
    may be state_in); o fp32 [T, Hv, Dv]; status an optional int32 device word."""
    _check(lib().moe_gdn_scan(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta),
                              _ptr(offsets), _ptr(state_in), _ptr(state_out), _ptr(o), _ptr(status),
                              _stream(stream)), "moe_gdn_scan")


def gdn_scan_timed(shape, q, k, v, gate, beta, offsets, state_in, state_out, o, events, status=None, stream=None):
    ev = (P * 2)(*events)
    _check(lib().moe_gdn_scan_timed(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta),
                                    _ptr(offsets), _ptr(state_in), _ptr(state_out), _ptr(o), _ptr(status), ev,
                                    _stream(stream)), "moe_gdn_scan_timed")


# ------------------------------------------------------- 8-bit KV cache ---

KV8_INT8, KV8_E4M3 = 0, 1


def kv8_shape(B, T, Hq, Hkv, D, L_max, block=64, format=KV8_INT8, q_stride=0, kv_stride=0) -> Kv8Shape:
    """A call over B sequences with T packed tokens in all. q_stride and
    kv_stride: elements between the tokens of q and of k_new, v_new (0:
    packed), for tokens that are column ranges of one projection's output."""
    return Kv8Shape(B, T, Hq, Hkv, D, L_max, block, format, q_stride, kv_stride)


def _kv8_refuse(where, what):
    raise MoeError(MOE_ERR_INVALID_ARG, where, what)


def _kv8_tensor(where, name, t, dev, dtype, dims, strides):
    """Refuses a tensor of the wrong type, sizes, strides (of dimensions longer
    than one) or device: what the C entry points cannot check. The wrappers
    call this only for a tensor that the usual one's quick test did not pass:
    at 0.5 us for each of a call's tensors it was a third of a short call."""
    if t.dtype is not dtype:
        _kv8_refuse(where, f"{name} is {t.dtype}, not {dtype}")
    if t.shape != dims:
        _kv8_refuse(where, f"{name} has shape {tuple(t.shape)}, not {dims}")
    if any(n > 1 and a != b for n, a, b in zip(dims, t.stride(), strides)) and t.numel() > 0:
        _kv8_refuse(where, f"{name} has strides {t.stride()}, not {strides}")
    if t.get_device() != dev:
        _kv8_refuse(where, f"{name} is on {t.device}, not on cuda:{dev}")
    return t.data_ptr()


_kv8_fields = struct.Struct("10i").unpack  # of a Kv8Shape
_BF16, _I32 = torch.bfloat16, torch.int32


class Kv8Cache:
    """An 8-bit KV cache: codes [B, Hkv, L_max, D] (uint8, or float8_e4m3fn
    for KV8_E4M3) and scales fp32 [B, Hkv, ceil(L_max / block)], contiguous, on
    one device. The tensors are checked here, once, and belong to the cache
    from then on (read them as .k, .v, .k_scale, .v_scale)."""

    __slots__ = ("_t", "_c", "_dims", "_nblk", "_e4m3", "_dev")

    def __init__(self, k, v, k_scale, v_scale):
        w = "Kv8Cache"
        if k.dim() != 4 or k_scale.dim() != 3 or k.dtype not in (torch.uint8, torch.float8_e4m3fn):
            _kv8_refuse(w, f"k is {k.dtype} {tuple(k.shape)}, k_scale {tuple(k_scale.shape)}: codes are uint8 or "
                           "float8_e4m3fn [B, Hkv, L_max, D], scales [B, Hkv, blocks]")
        dims, dev = tuple(k.shape), k.get_device()
        B, H, L, D = dims
        nblk = k_scale.shape[2]
        strides, sdims, sstrides = (H * L * D, L * D, D, 1), (B, H, nblk), (H * nblk, nblk, 1)
        self._c = Kv8CacheC(_kv8_tensor(w, "k", k, dev, k.dtype, dims, strides),
                            _kv8_tensor(w, "v", v, dev, k.dtype, dims, strides),
                            _kv8_tensor(w, "k_scale", k_scale, dev, torch.float32, sdims, sstrides),
                            _kv8_tensor(w, "v_scale", v_scale, dev, torch.float32, sdims, sstrides))
        self._t = (k, v, k_scale, v_scale)
        self._dims, self._nblk, self._e4m3, self._dev = dims, nblk, k.dtype is torch.float8_e4m3fn, dev

    k = property(lambda self: self._t[0])
    v = property(lambda self: self._t[1])
    k_scale = property(lambda self: self._t[2])
    v_scale = property(lambda self: self._t[3])

    def _device(self, where, shape):
        """Refuses a cache that is not one of `shape` on the current device; as
        _kv8_tensor, called where the wrapper's quick test did not pass."""
        if self._dims != (shape.B, shape.Hkv, shape.L_max, shape.D) or (
                self._nblk != -(-shape.L_max // max(shape.block, 1))) or (self._e4m3 and shape.format != KV8_E4M3):
            _kv8_refuse(where, f"the cache holds {self._t[0].dtype} codes {self._dims} in {self._nblk} blocks, the "
                               "shape says otherwise")
        if self._dev != torch.cuda.current_device():
            _kv8_refuse(where, f"the cache is on {self._t[0].device}, not on the current device")


def kv8_alloc_cache(shape: Kv8Shape, device) -> Kv8Cache:
    """An empty cache for `shape` (its contents need no initialisation)."""
    dt = torch.float8_e4m3fn if shape.format == KV8_E4M3 else torch.uint8
    codes = [torch.empty(shape.B, shape.Hkv, shape.L_max, shape.D, dtype=dt, device=device) for _ in range(2)]
    nblk = -(-shape.L_max // shape.block)
    return Kv8Cache(*codes, *[torch.empty(shape.B, shape.Hkv, nblk, device=device) for _ in range(2)])


# torch.cuda.current_device() and the handle of torch.cuda.current_stream(),
# without looking whether CUDA is up (the cache is on it) and a Stream object.
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def kv8_write(shape, k_new, v_new, offsets, starts, cache: Kv8Cache, status=None, stream=None):
    """moe_kv8_write: quantises k_new, v_new bf16 [T, Hkv, D] into `cache`;
    sequence b's tokens offsets[b] .. offsets[b+1]-1 go to its positions
    starts[b] .. (int32 [B+1] and [B]). status: an optional zeroed int32
    device word."""
    w = "moe_kv8_write"
    B, T, _, H, D, L, block, fmt, _, stride = _kv8_fields(shape)
    dev, dims, strides = cache._dev, (T, H, D), (stride or H * D, D, 1)
    if not (cache._dims == (B, H, L, D) and 0 <= cache._nblk * block - L < block and (fmt or not cache._e4m3)
            and dev >= 0 and _current_device() == dev):
        cache._device(w, shape)
    if not (k_new.dtype is _BF16 and k_new.shape == dims and k_new.stride() == strides and k_new.get_device() == dev):
        _kv8_tensor(w, "k_new", k_new, dev, _BF16, dims, strides)
    if not (v_new.dtype is _BF16 and v_new.shape == dims and v_new.stride() == strides and v_new.get_device() == dev):
        _kv8_tensor(w, "v_new", v_new, dev, _BF16, dims, strides)
    if not (offsets.dtype is _I32 and offsets.shape == (B + 1,) and offsets.is_contiguous()
            and offsets.get_device() == dev):
        _kv8_tensor(w, "offsets", offsets, dev, _I32, (B + 1,), (1,))
    if not (starts.dtype is _I32 and starts.shape == (B,) and starts.is_contiguous() and starts.get_device() == dev):
        _kv8_tensor(w, "starts", starts, dev, _I32, (B,), (1,))
    rc = lib().moe_kv8_write(shape, k_new.data_ptr(), v_new.data_ptr(), offsets.data_ptr(), starts.data_ptr(), cache._c,
                             None if status is None else _kv8_tensor(w, "status", status, dev, _I32, (1,), (1,)),
                             _current_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc, w)


def kv8_read(shape, cache: Kv8Cache, offsets, starts, k_out, v_out, status=None, stream=None):
    """moe_kv8_read: positions starts[b] .. of every sequence as bf16, packed
    in k_out, v_out [T, Hkv, D]."""
    w = "moe_kv8_read"
    B, T, _, H, D, L, block, fmt, _, _ = _kv8_fields(shape)
    dev, dims = cache._dev, (T, H, D)
    if not (cache._dims == (B, H, L, D) and 0 <= cache._nblk * block - L < block and (fmt or not cache._e4m3)
            and dev >= 0 and _current_device() == dev):
        cache._device(w, shape)
    if not (offsets.dtype is _I32 and offsets.shape == (B + 1,) and offsets.is_contiguous()
            and offsets.get_device() == dev):
        _kv8_tensor(w, "offsets", offsets, dev, _I32, (B + 1,), (1,))
    if not (starts.dtype is _I32 and starts.shape == (B,) and starts.is_contiguous() and starts.get_device() == dev):
        _kv8_tensor(w, "starts", starts, dev, _I32, (B,), (1,))
    if not (k_out.dtype is _BF16 and k_out.shape == dims and k_out.is_contiguous() and k_out.get_device() == dev):
        _kv8_tensor(w, "k_out", k_out, dev, _BF16, dims, (H * D, D, 1))
    if not (v_out.dtype is _BF16 and v_out.shape == dims and v_out.is_contiguous() and v_out.get_device() == dev):
        _kv8_tensor(w, "v_out", v_out, dev, _BF16, dims, (H * D, D, 1))
    rc = lib().moe_kv8_read(shape, cache._c, offsets.data_ptr(), starts.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
                            None if status is None else _kv8_tensor(w, "status", status, dev, _I32, (1,), (1,)),
                            _current_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc, w)


def kv8_workspace_bytes(shape: Kv8Shape) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_kv8_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_kv8_workspace_bytes")
    return n.value


def kv8_alloc_workspace(shape: Kv8Shape, device) -> torch.Tensor:
    return torch.empty(kv8_workspace_bytes(shape), dtype=torch.uint8, device=device)


def kv8_attn(shape, q, cache: Kv8Cache, offsets, lens, o, workspace, scale=None, stream=None):
    """moe_kv8_attn: q bf16 [T, Hq, D], the last tokens of every sequence
    (offsets int32 [B+1]) over its lens[b] cached positions (int32 [B]); o bf16
    [T, Hq, D]. The workspace's first int32 is the call's device status word."""
    w = "moe_kv8_attn"
    B, T, H, Hkv, D, L, block, fmt, stride, _ = _kv8_fields(shape)
    dev, dims, strides, n = cache._dev, (T, H, D), (stride or H * D, D, 1), workspace.numel()
    if not (cache._dims == (B, Hkv, L, D) and 0 <= cache._nblk * block - L < block and (fmt or not cache._e4m3)
            and dev >= 0 and _current_device() == dev):
        cache._device(w, shape)
    if not (q.dtype is _BF16 and q.shape == dims and q.stride() == strides and q.get_device() == dev):
        _kv8_tensor(w, "q", q, dev, _BF16, dims, strides)
    if not (offsets.dtype is _I32 and offsets.shape == (B + 1,) and offsets.is_contiguous()
            and offsets.get_device() == dev):
        _kv8_tensor(w, "offsets", offsets, dev, _I32, (B + 1,), (1,))
    if not (lens.dtype is _I32 and lens.shape == (B,) and lens.is_contiguous() and lens.get_device() == dev):
        _kv8_tensor(w, "lens", lens, dev, _I32, (B,), (1,))
    if not (o.dtype is _BF16 and o.shape == dims and o.is_contiguous() and o.get_device() == dev):
        _kv8_tensor(w, "o", o, dev, _BF16, dims, (H * D, D, 1))
    if not (workspace.dtype is torch.uint8 and workspace.is_contiguous() and workspace.get_device() == dev):
        _kv8_tensor(w, "workspace", workspace, dev, torch.uint8, (n,), (1,))
    rc = lib().moe_kv8_attn(shape, q.data_ptr(), cache._c, offsets.data_ptr(), lens.data_ptr(),
                            D ** -0.5 if scale is None else scale, o.data_ptr(), workspace.data_ptr(), n,
                            _current_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc, w)


def kv8_attn_test_stall(shape, q, cache: Kv8Cache, offsets, lens, o, workspace, stalled_block: int, timeout_ns: int,
                        scale=None, stream=None):
    """moe_kv8_attn_test_stall: kv8_attn with one grid block that never brings
    its operands and a short device timeout (test only)."""
    _check(lib().moe_kv8_attn_test_stall(shape, _ptr(q), cache._c, _ptr(offsets), _ptr(lens),
                                         shape.D ** -0.5 if scale is None else scale, _ptr(o), _ptr(workspace),
                                         workspace.numel(), int(stalled_block), int(timeout_ns), _stream(stream)),
           "moe_kv8_attn_test_stall")
