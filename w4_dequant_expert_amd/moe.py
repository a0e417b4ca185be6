"""Python binding of libmoe_w4.so: argument marshalling only.

Every call goes straight to the C ABI declared in include/moe_w4.h,
include/gdn_scan.h and include/moe_block.h; all of the layer's arithmetic runs
in the HIP kernels.  PyTorch is used only to allocate
device memory and to name the stream the kernels are enqueued on.  If the
library is missing the import fails: there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_w4.so")

MOE_OK, MOE_EINVAL, MOE_EALIGN, MOE_EWS, MOE_EDEVICE, MOE_ELAUNCH = 0, -1, -2, -3, -4, -5
NO_ALLOC_WS_BYTES = 4 << 20   # MOE_NO_ALLOC_WS_BYTES
STATUS_NAN_LOGIT, STATUS_BAD_INDEX, STATUS_BLOCK_OVERFLOW = 1, 2, 4

EXPORTED = ("moe_abi_version", "moe_strerror", "moe_max_blocks", "moe_route_ws_bytes", "moe_route",
            "moe_route_no_alloc",
            "moe_w4_gate_up", "moe_w4_down", "moe_grouped_w4_ffn", "moe_shared_w4_ffn",
            "moe_routed_w4_ffn", "moe_combine", "moe_w4_ffn_combine", "moe_w4_dequant",
            "moe_w4_dequant_packed", "moe_w4_packed_bytes",
            "moe_w4_pack", "moe_read_probe", "moe_mfma_probe", "gdn_scan",
            "gdn_scan_chunked", "gdn_scan_chunked_ws_bytes", "moe_add_rmsnorm",
            "moe_add_rmsnorm_backward", "moe_add_rmsnorm_backward_ws_bytes", "moe_q8_quantize",
            "moe_q8_matmul", "moe_q8_gate_up", "moe_q8_down", "moe_dispatch_rows",
            "moe_dispatch_rows_backward", "moe_combine_rows", "moe_combine_rows_backward")

ELEM_F32, ELEM_BF16, ELEM_F16 = 0, 1, 2   # MOE_ELEM_*
NORM_MAX_T, NORM_MAX_H = 1 << 24, 16384   # moe_norm_dims
ELEM: dict = {}   # torch dtype -> MOE_ELEM_*, filled when the library is loaded
# the torch types that the arrays of each kind may have, and (bytes, types) of each row type; set with ELEM
_F32 = _I8 = _BF16 = ()
_ROW_TYPES: dict = {}
_UNKNOWN = (0, None)   # a row type that the C side refuses


class GdnDims(ctypes.Structure):
    """gdn_dims of include/gdn_scan.h."""
    _fields_ = [("T", ctypes.c_int32), ("n_k_heads", ctypes.c_int32), ("n_v_heads", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32)]


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "E", "k", "n_shared", "tile_m_max",
                                              "tile_gran")]


class Bank(ctypes.Structure):
    """Packed bank: gate/up and down matrices of n experts."""
    _fields_ = [("gu", ctypes.c_void_p), ("dn", ctypes.c_void_p)]


class RouteOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "counts", "offsets",
                                               "sorted_slot", "slot_pos", "blocks", "n_blocks",
                                               "logits", "status", "ws")] + [("ws_bytes", ctypes.c_size_t)]


class NormDims(ctypes.Structure):
    """moe_norm_dims of include/moe_block.h; type is one of ELEM_*."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("type", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class Q8Dims(ctypes.Structure):
    """moe_q8_dims of include/moe_block.h; type is the output's."""
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "type")]


class Q8Bank(ctypes.Structure):
    """8-bit bank: gate/up and down matrices of n experts and their channel scales."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("gu", "gu_s", "dn", "dn_s")]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {strerror(code)} (code {code})")
        self.code = code


_lib = None
# set with _lib
_torch = _get_device = _raw_stream = None
_cuda_ready = False


def lib():
    global _lib, _torch, _get_device, _raw_stream, _F32, _I8, _BF16
    if _lib is None:
        # torch ships its own HIP runtime.  Import it first so that loading the
        # library resolves libamdhip64.so.7 to that same runtime; loading the
        # library first would bring a second HIP runtime into the process, and
        # torch's streams and memory would then be foreign to our kernels.
        import torch  # noqa: F401
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it first "
                              "(python __graft_entry__.py, or python w4_dequant_expert_amd/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp = ctypes.c_void_p
        L.moe_abi_version.restype = ctypes.c_int
        L.moe_abi_version.argtypes = []
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_strerror.argtypes = [ctypes.c_int]
        L.moe_max_blocks.restype = ctypes.c_int32
        L.moe_max_blocks.argtypes = [P(Dims)]
        L.moe_route_ws_bytes.restype = ctypes.c_size_t
        L.moe_route_ws_bytes.argtypes = [P(Dims)]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [P(Dims), vp, vp, vp, P(RouteOut), vp]
        L.moe_route_no_alloc.restype = ctypes.c_int
        L.moe_route_no_alloc.argtypes = [P(Dims), vp, vp, vp, P(RouteOut), vp]
        L.moe_w4_gate_up.restype = ctypes.c_int
        L.moe_w4_gate_up.argtypes = [P(Dims), vp, P(RouteOut), P(Bank), P(Bank), vp, vp]
        L.moe_w4_down.restype = ctypes.c_int
        L.moe_w4_down.argtypes = [P(Dims), P(RouteOut), P(Bank), P(Bank), vp, vp, vp]
        L.moe_grouped_w4_ffn.restype = ctypes.c_int
        L.moe_grouped_w4_ffn.argtypes = [P(Dims), vp, P(RouteOut), P(Bank), P(Bank), vp, vp, vp]
        L.moe_shared_w4_ffn.restype = ctypes.c_int
        L.moe_shared_w4_ffn.argtypes = [P(Dims), vp, P(Bank), vp, vp, vp]
        L.moe_routed_w4_ffn.restype = ctypes.c_int
        L.moe_routed_w4_ffn.argtypes = [P(Dims), vp, P(RouteOut), P(Bank), vp, vp, vp]
        L.moe_combine.restype = ctypes.c_int
        L.moe_combine.argtypes = [P(Dims), P(RouteOut), vp, vp, vp]
        L.moe_w4_ffn_combine.restype = ctypes.c_int
        L.moe_w4_ffn_combine.argtypes = [P(Dims), vp, P(RouteOut), P(Bank), P(Bank), vp, vp, vp, vp]
        L.moe_w4_dequant.restype = ctypes.c_int
        L.moe_w4_dequant.argtypes = [ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp, vp]
        L.moe_w4_dequant_packed.restype = ctypes.c_int
        L.moe_w4_dequant_packed.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                            ctypes.c_int32, vp, vp, vp]
        L.moe_read_probe.restype = ctypes.c_int
        L.moe_read_probe.argtypes = [vp, ctypes.c_size_t, vp, ctypes.c_int32, vp]
        L.moe_w4_packed_bytes.restype = ctypes.c_size_t
        L.moe_w4_packed_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
        L.moe_w4_pack.restype = ctypes.c_int
        L.moe_w4_pack.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  vp, vp, vp, vp, vp]
        L.moe_mfma_probe.restype = ctypes.c_int
        L.moe_mfma_probe.argtypes = [ctypes.c_int32, ctypes.c_int32, vp, vp]
        L.gdn_scan_chunked.restype = ctypes.c_int
        L.gdn_scan_chunked.argtypes = [P(GdnDims), vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.gdn_scan_chunked_ws_bytes.restype = ctypes.c_size_t
        L.gdn_scan_chunked_ws_bytes.argtypes = [P(GdnDims)]
        L.gdn_scan.restype = ctypes.c_int
        L.gdn_scan.argtypes = [P(GdnDims), vp, vp, vp, vp, vp, vp, vp, vp, vp]
        i32, size = ctypes.c_int32, ctypes.c_size_t
        L.moe_add_rmsnorm.restype = ctypes.c_int
        L.moe_add_rmsnorm.argtypes = [P(NormDims), vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_add_rmsnorm_backward_ws_bytes.restype = size
        L.moe_add_rmsnorm_backward_ws_bytes.argtypes = [P(NormDims)]
        L.moe_add_rmsnorm_backward.restype = ctypes.c_int
        L.moe_add_rmsnorm_backward.argtypes = [P(NormDims), vp, vp, vp, vp, vp, vp, vp, size, vp]
        L.moe_q8_quantize.restype = ctypes.c_int
        L.moe_q8_quantize.argtypes = [P(NormDims), vp, vp, vp, vp]
        L.moe_q8_matmul.restype = ctypes.c_int
        L.moe_q8_matmul.argtypes = [P(Q8Dims), vp, vp, vp, vp, vp, vp]
        L.moe_q8_gate_up.restype = ctypes.c_int
        L.moe_q8_gate_up.argtypes = [P(Dims), vp, vp, P(RouteOut), P(Q8Bank), P(Q8Bank), vp, vp]
        L.moe_q8_down.restype = ctypes.c_int
        L.moe_q8_down.argtypes = [P(Dims), P(RouteOut), P(Q8Bank), P(Q8Bank), vp, vp, vp, vp]
        for name in ("moe_dispatch_rows", "moe_dispatch_rows_backward", "moe_combine_rows"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [P(Dims), i32, vp, P(RouteOut), vp, vp]
        L.moe_combine_rows_backward.restype = ctypes.c_int
        L.moe_combine_rows_backward.argtypes = [P(Dims), i32, vp, vp, P(RouteOut), vp, vp, vp]
        ELEM.update({torch.float32: ELEM_F32, torch.bfloat16: ELEM_BF16, torch.float16: ELEM_F16})
        bits = (torch.int16, torch.uint16)
        _F32, _I8, _BF16 = (torch.float32,), (torch.int8,), (torch.bfloat16, *bits)
        _ROW_TYPES.update({ELEM_F32: (4, _F32), ELEM_BF16: (2, _BF16), ELEM_F16: (2, (torch.float16, *bits))})
        _get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _lib, _torch = L, torch
    return _lib


def strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _ptr(t):
    """Device address of a torch tensor (None -> NULL); ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _device() -> int:
    """The current GPU."""
    if not _cuda_ready:
        _init_cuda()
    return _get_device()


def _init_cuda():
    global _cuda_ready
    if not _torch.cuda.is_initialized():
        _torch.cuda.init()
    _cuda_ready = True


def _after_fork():
    global _cuda_ready
    _cuda_ready = False   # torch then refuses the child's use of the GPU


os.register_at_fork(after_in_child=_after_fork)


def _stream(stream, device=None):
    if stream is None:
        # the handle alone: building a stream object costs more than a small launch
        return _raw_stream(_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# --------------------------------------------------------------------- the C ABI

def moe_abi_version() -> int:
    return lib().moe_abi_version()


def moe_max_blocks(d: Dims) -> int:
    return lib().moe_max_blocks(ctypes.byref(d))


def moe_route_ws_bytes(d: Dims) -> int:
    return lib().moe_route_ws_bytes(ctypes.byref(d))


def moe_route(d: Dims, x, w_router, logit_bias, out: RouteOut, stream=None):
    _check(lib().moe_route(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(logit_bias),
                           ctypes.byref(out), _stream(stream)), "moe_route")


def moe_route_no_alloc(d: Dims, x, w_router, logit_bias, out: RouteOut, stream=None):
    _check(lib().moe_route_no_alloc(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                    ctypes.byref(out), _stream(stream)), "moe_route_no_alloc")


def moe_w4_gate_up(d: Dims, x, out: RouteOut, routed: Bank, shared, h, stream=None):
    _check(lib().moe_w4_gate_up(ctypes.byref(d), _ptr(x), ctypes.byref(out), ctypes.byref(routed),
                                ctypes.byref(shared) if shared is not None else None, _ptr(h),
                                _stream(stream)), "moe_w4_gate_up")


def moe_w4_down(d: Dims, out: RouteOut, routed: Bank, shared, h, y_slots, stream=None):
    _check(lib().moe_w4_down(ctypes.byref(d), ctypes.byref(out), ctypes.byref(routed),
                             ctypes.byref(shared) if shared is not None else None, _ptr(h),
                             _ptr(y_slots), _stream(stream)), "moe_w4_down")


def moe_grouped_w4_ffn(d: Dims, x, out: RouteOut, routed: Bank, shared, h, y_slots, stream=None):
    _check(lib().moe_grouped_w4_ffn(ctypes.byref(d), _ptr(x), ctypes.byref(out),
                                    ctypes.byref(routed),
                                    ctypes.byref(shared) if shared is not None else None,
                                    _ptr(h), _ptr(y_slots), _stream(stream)), "moe_grouped_w4_ffn")


def moe_shared_w4_ffn(d: Dims, x, shared: Bank, h, y_slots, stream=None):
    _check(lib().moe_shared_w4_ffn(ctypes.byref(d), _ptr(x), ctypes.byref(shared), _ptr(h),
                                   _ptr(y_slots), _stream(stream)), "moe_shared_w4_ffn")


def moe_routed_w4_ffn(d: Dims, x, out: RouteOut, routed: Bank, h, y_slots, stream=None):
    _check(lib().moe_routed_w4_ffn(ctypes.byref(d), _ptr(x), ctypes.byref(out), ctypes.byref(routed),
                                   _ptr(h), _ptr(y_slots), _stream(stream)), "moe_routed_w4_ffn")


def moe_combine(d: Dims, out: RouteOut, y_slots, y, stream=None):
    _check(lib().moe_combine(ctypes.byref(d), ctypes.byref(out), _ptr(y_slots), _ptr(y),
                             _stream(stream)), "moe_combine")


def moe_w4_ffn_combine(d: Dims, x, out: RouteOut, routed: Bank, shared, h, y_slots, y, stream=None):
    _check(lib().moe_w4_ffn_combine(ctypes.byref(d), _ptr(x), ctypes.byref(out), ctypes.byref(routed),
                                    ctypes.byref(shared) if shared is not None else None,
                                    _ptr(h), _ptr(y_slots), _ptr(y), _stream(stream)),
           "moe_w4_ffn_combine")


def moe_w4_dequant(rows: int, K: int, q, s, b, out, stream=None):
    _check(lib().moe_w4_dequant(rows, K, _ptr(q), _ptr(s), _ptr(b), _ptr(out), _stream(stream)),
           "moe_w4_dequant")


def moe_w4_dequant_packed(n: int, rows: int, K: int, gate_up: bool, packed, out, stream=None):
    _check(lib().moe_w4_dequant_packed(n, rows, K, 1 if gate_up else 0, _ptr(packed), _ptr(out),
                                       _stream(stream)), "moe_w4_dequant_packed")


def moe_read_probe(src, nbytes: int, sink, workgroups: int, stream=None):
    _check(lib().moe_read_probe(_ptr(src), nbytes, _ptr(sink), workgroups, _stream(stream)),
           "moe_read_probe")


def moe_mfma_probe(workgroups: int, iters: int, sink, stream=None):
    _check(lib().moe_mfma_probe(workgroups, iters, _ptr(sink), _stream(stream)), "moe_mfma_probe")


def moe_w4_packed_bytes(rows: int, K: int) -> int:
    return lib().moe_w4_packed_bytes(rows, K)


def moe_w4_pack(n: int, rows: int, K: int, gate_up: bool, q, s, b, packed, stream=None):
    _check(lib().moe_w4_pack(n, rows, K, 1 if gate_up else 0, _ptr(q), _ptr(s), _ptr(b),
                             _ptr(packed), _stream(stream)), "moe_w4_pack")


def gdn_scan(d: GdnDims, q, k, v, g, beta, state_in, state_out, o, stream=None):
    """Gated DeltaNet scan of include/gdn_scan.h (device tensors or raw addresses)."""
    _check(lib().gdn_scan(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                          _ptr(state_in), _ptr(state_out), _ptr(o), _stream(stream)), "gdn_scan")


def gdn_scan_chunked_ws_bytes(d: GdnDims) -> int:
    return lib().gdn_scan_chunked_ws_bytes(ctypes.byref(d))


def gdn_scan_chunked(d: GdnDims, q, k, v, g, beta, state_in, state_out, o, ws, ws_bytes: int,
                     stream=None):
    """Chunked Gated DeltaNet scan of include/gdn_scan.h."""
    _check(lib().gdn_scan_chunked(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(state_in), _ptr(state_out), _ptr(o), _ptr(ws), ws_bytes,
                                  _stream(stream)), "gdn_scan_chunked")


# ------------------------------------------- around the expert layer (include/moe_block.h)

def _arg(t, nbytes: int, what: str, device: int, types=None):
    """Address of a dense array of at least nbytes on `device` (None -> NULL; raw addresses pass).

    The C side cannot see sizes, strides or types, so tensors that are strided,
    too small, off the current device or of another type than `types` (None:
    any; 16-bit rows may come as the integers of their bits) are refused here.
    The type of an array that is not looked at (nbytes 0) does not count."""
    if t is None or type(t) is int:
        return t
    if (t.nbytes < nbytes or not t.is_contiguous() or t.get_device() != device or
            (types is not None and nbytes and t.dtype not in types)):
        raise ValueError(f"{what}: a contiguous tensor of at least {nbytes} bytes on GPU {device} is needed"
                         f"{'' if types is None else ' of ' + ' or '.join(map(str, types))}, got "
                         f"{tuple(t.shape)} {t.dtype} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def moe_add_rmsnorm(d: NormDims, x, res, weight, sum, y, yq=None, ys=None, stream=None):
    """Residual addition and RMS norm (any of res, sum, y, yq with ys may be None)."""
    dev = _device()
    n = d.T * d.H
    size, typ = _ROW_TYPES.get(d.type, _UNKNOWN)
    row = n * size
    _check(_lib.moe_add_rmsnorm(d, _arg(x, row, "x", dev, typ), _arg(res, row, "res", dev, typ),
                                _arg(weight, 4 * d.H, "weight", dev, _F32), _arg(sum, row, "sum", dev, typ),
                                _arg(y, row, "y", dev, typ), _arg(yq, n, "yq", dev, _I8),
                                _arg(ys, 4 * d.T, "ys", dev, _F32), _stream(stream, dev)), "moe_add_rmsnorm")


def moe_add_rmsnorm_backward_ws_bytes(d: NormDims) -> int:
    return _lib.moe_add_rmsnorm_backward_ws_bytes(d)


def moe_add_rmsnorm_backward(d: NormDims, sum, weight, dy, dsum, dx, dweight, ws, ws_bytes: int,
                             stream=None):
    """Gradients of moe_add_rmsnorm (dsum and dweight may be None)."""
    dev = _device()
    size, typ = _ROW_TYPES.get(d.type, _UNKNOWN)
    row = d.T * d.H * size
    _check(_lib.moe_add_rmsnorm_backward(
        d, _arg(sum, row, "sum", dev, typ), _arg(weight, 4 * d.H, "weight", dev, _F32),
        _arg(dy, row, "dy", dev, typ), _arg(dsum, row, "dsum", dev, typ), _arg(dx, row, "dx", dev, typ),
        _arg(dweight, 4 * d.H, "dweight", dev, _F32), _arg(ws, ws_bytes, "ws", dev), ws_bytes,
        _stream(stream, dev)), "moe_add_rmsnorm_backward")


def moe_q8_quantize(d: NormDims, x, xq, xs, stream=None):
    """Rows to int8 with a scale per row."""
    dev = _device()
    n = d.T * d.H
    size, typ = _ROW_TYPES.get(d.type, _UNKNOWN)
    _check(_lib.moe_q8_quantize(d, _arg(x, n * size, "x", dev, typ), _arg(xq, n, "xq", dev, _I8),
                                _arg(xs, 4 * d.T, "xs", dev, _F32), _stream(stream, dev)),
           "moe_q8_quantize")


def moe_q8_matmul(d: Q8Dims, xq, xs, wq, ws, out, stream=None):
    """Dense product of 8-bit integers with token and channel scales."""
    dev = _device()
    size, typ = _ROW_TYPES.get(d.type, _UNKNOWN)
    _check(_lib.moe_q8_matmul(d, _arg(xq, d.M * d.K, "xq", dev, _I8), _arg(xs, 4 * d.M, "xs", dev, _F32),
                              _arg(wq, d.N * d.K, "wq", dev, _I8), _arg(ws, 4 * d.N, "ws", dev, _F32),
                              _arg(out, d.M * d.N * size, "out", dev, typ), _stream(stream, dev)),
           "moe_q8_matmul")


def _rows_of(d: Dims) -> int:
    return d.T * (d.k + d.n_shared)


def moe_q8_gate_up(d: Dims, xq, xs, out: RouteOut, routed: Q8Bank, shared, h, stream=None):
    dev = _device()
    _check(_lib.moe_q8_gate_up(d, _arg(xq, d.T * d.H, "xq", dev, _I8), _arg(xs, 4 * d.T, "xs", dev, _F32),
                               out, routed, shared,
                               _arg(h, 2 * _rows_of(d) * d.I, "h", dev, _BF16), _stream(stream, dev)),
           "moe_q8_gate_up")


def moe_q8_down(d: Dims, out: RouteOut, routed: Q8Bank, shared, hq, hs, y_slots, stream=None):
    dev = _device()
    rows = _rows_of(d)
    _check(_lib.moe_q8_down(d, out, routed, shared,
                            _arg(hq, rows * d.I, "hq", dev, _I8), _arg(hs, 4 * rows, "hs", dev, _F32),
                            _arg(y_slots, 2 * rows * d.H, "y_slots", dev, _BF16), _stream(stream, dev)),
           "moe_q8_down")


def moe_dispatch_rows(d: Dims, elem: int, x, out: RouteOut, rows, stream=None):
    """Token rows into moe_route's order (elem: one of ELEM_*)."""
    dev = _device()
    size, typ = _ROW_TYPES.get(elem, _UNKNOWN)
    e = size * d.H
    _check(_lib.moe_dispatch_rows(d, elem, _arg(x, d.T * e, "x", dev, typ), out,
                                  _arg(rows, _rows_of(d) * e, "rows", dev, typ), _stream(stream, dev)),
           "moe_dispatch_rows")


def moe_dispatch_rows_backward(d: Dims, elem: int, drows, out: RouteOut, dx, stream=None):
    dev = _device()
    size, typ = _ROW_TYPES.get(elem, _UNKNOWN)
    e = size * d.H
    _check(_lib.moe_dispatch_rows_backward(d, elem, _arg(drows, _rows_of(d) * e, "drows", dev, typ),
                                           out, _arg(dx, d.T * e, "dx", dev, typ),
                                           _stream(stream, dev)), "moe_dispatch_rows_backward")


def moe_combine_rows(d: Dims, elem: int, rows, out: RouteOut, y, stream=None):
    """moe_combine for any row type."""
    dev = _device()
    size, typ = _ROW_TYPES.get(elem, _UNKNOWN)
    e = size * d.H
    _check(_lib.moe_combine_rows(d, elem, _arg(rows, _rows_of(d) * e, "rows", dev, typ),
                                 out, _arg(y, d.T * e, "y", dev, typ), _stream(stream, dev)),
           "moe_combine_rows")


def moe_combine_rows_backward(d: Dims, elem: int, dy, rows, out: RouteOut, drows, dtopk_w,
                              stream=None):
    """Gradients of the combine (dtopk_w None: rows is not read and may be None)."""
    dev = _device()
    size, typ = _ROW_TYPES.get(elem, _UNKNOWN)
    e = size * d.H
    _check(_lib.moe_combine_rows_backward(d, elem, _arg(dy, d.T * e, "dy", dev, typ),
                                          _arg(rows, _rows_of(d) * e, "rows", dev, typ), out,
                                          _arg(drows, _rows_of(d) * e, "drows", dev, typ),
                                          _arg(dtopk_w, 4 * d.T * d.k, "dtopk_w", dev, _F32),
                                          _stream(stream, dev)), "moe_combine_rows_backward")


# --------------------------------------------------------------------- device buffers

def make_dims(T, H, I, E, k, n_shared, tile_m_max=128, tile_gran=16) -> Dims:
    return Dims(T, H, I, E, k, n_shared, tile_m_max, tile_gran)


def _dev(a: np.ndarray, device):
    import torch
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


class DeviceBank:
    """An expert bank resident in device memory in the packed streaming layout.

    The canonical-layout arrays (numpy, as in a checkpoint) are uploaded once,
    repacked on the device by moe_w4_pack, and released.
    """

    CANON = ("gu_q", "gu_s", "gu_b", "dn_q", "dn_s", "dn_b")

    def __init__(self, bank: dict, device="cuda"):
        import torch
        n, two_i, half_h = bank["gu_q"].shape
        H = 2 * half_h
        I = two_i // 2
        self.n, self.H, self.I = n, H, I
        canon = {k: _dev(bank[k], device) for k in self.CANON}
        gu = torch.empty((n, moe_w4_packed_bytes(2 * I, H)), dtype=torch.uint8, device=device)
        dn = torch.empty((n, moe_w4_packed_bytes(H, I)), dtype=torch.uint8, device=device)
        moe_w4_pack(n, 2 * I, H, True, canon["gu_q"], canon["gu_s"], canon["gu_b"], gu)
        moe_w4_pack(n, H, I, False, canon["dn_q"], canon["dn_s"], canon["dn_b"], dn)
        torch.cuda.current_stream().synchronize()
        del canon
        self.t = {"gu": gu, "dn": dn}
        self.c = Bank(gu.data_ptr(), dn.data_ptr())

    @classmethod
    def from_tensors(cls, tensors: dict, n, H, I):
        self = cls.__new__(cls)
        self.t = tensors
        self.n, self.H, self.I = n, H, I
        self.c = Bank(tensors["gu"].data_ptr(), tensors["dn"].data_ptr())
        return self

    def clone(self):
        return DeviceBank.from_tensors({k: v.clone() for k, v in self.t.items()}, self.n, self.H,
                                       self.I)

    def nbytes(self) -> int:
        return sum(v.numel() * v.element_size() for v in self.t.values())


def _check_q8_widths(H, I):
    if not (0 < H <= NORM_MAX_H and 0 < I <= NORM_MAX_H):
        raise ValueError(f"H={H}, I={I}: rows are quantised at up to {NORM_MAX_H} elements")


def _pieces(n: int, rows: int, K: int):
    """Slices of n matrices of rows x K that one call takes: the quantiser 2^24 rows, the dequantiser
    fewer than 2^32 groups of eight weights (a thread each, 256 a workgroup)."""
    step = max(1, min(NORM_MAX_T // rows, (2 ** 35 - 2 ** 11) // (rows * K)))
    return [slice(lo, min(lo + step, n)) for lo in range(0, n, step)]


class DeviceBankQ8:
    """An expert bank resident in device memory in 8 bits (moe_q8_bank).

    gu [n][2I][H] (gate rows, then up rows) and dn [n][H][I] are float device
    tensors, H and I at most NORM_MAX_H; each output channel is quantised once by
    moe_q8_quantize.
    """

    def __init__(self, gu, dn):
        import torch
        n, two_i, H = gu.shape
        self.n, self.H, self.I = n, H, two_i // 2
        if two_i % 2:
            raise ValueError(f"gu has {two_i} rows an expert: gate and up rows come in pairs")
        _check_q8_widths(H, self.I)
        if dn.shape != (n, H, self.I):
            raise ValueError(f"dn has shape {tuple(dn.shape)}, not {(n, H, self.I)}")
        gq, gs = self._quantize(gu)
        dq, ds = self._quantize(dn)
        torch.cuda.current_stream().synchronize()   # the bank may be used on any stream from here on
        self.t = {"gu": gq, "gu_s": gs, "dn": dq, "dn_s": ds}
        self.c = Q8Bank(*[self.t[k].data_ptr() for k in ("gu", "gu_s", "dn", "dn_s")])

    @classmethod
    def from_w4(cls, bank: dict, device="cuda"):
        """From the canonical 4-bit arrays of a checkpoint (as DeviceBank takes them)."""
        import torch
        out = []
        for half in ("gu", "dn"):
            q, s, b = (_dev(bank[f"{half}_{p}"], device) for p in "qsb")
            n, rows, half_k = q.shape
            w = torch.empty((n, rows, 2 * half_k), dtype=torch.bfloat16, device=device)
            # what the dequantiser reads and writes lies on the current device, and is all there
            dev, groups = _device(), n * rows * (half_k // 32)
            _arg(q, 1, f"{half}_q", dev, (torch.uint8,))
            _arg(s, 2 * groups, f"{half}_s", dev, _BF16)
            _arg(b, 2 * groups, f"{half}_b", dev, _BF16)
            for e in _pieces(n, rows, 2 * half_k):
                moe_w4_dequant(w[e].shape[0] * rows, 2 * half_k, q[e], s[e], b[e], w[e])
            out.append(w)
        return cls(*out)

    @staticmethod
    def _quantize(w):
        import torch
        n, rows, K = w.shape
        q = torch.empty((n, rows, K), dtype=torch.int8, device=w.device)
        s = torch.empty((n, rows), dtype=torch.float32, device=w.device)
        for e in _pieces(n, rows, K):
            part = w[e].contiguous()
            moe_q8_quantize(NormDims(part.shape[0] * rows, K, ELEM[w.dtype], 0.0), part, q[e], s[e])
        return q, s

    def nbytes(self) -> int:
        return sum(v.numel() * v.element_size() for v in self.t.values())

    def __repr__(self):
        return f"DeviceBankQ8 of {self.n} experts, H {self.H}, I {self.I} on {self.t['gu'].device}"


class RouteTables:
    """Device arrays for every routing output of one layer call of up to T tokens."""

    def __init__(self, d: Dims, device="cuda", export_logits=True):
        import torch
        T, E, k = d.T, d.E, d.k
        i32 = dict(dtype=torch.int32, device=device)
        self.d = d
        self.topk_idx = torch.empty((T, k), **i32)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.counts = torch.empty((E,), **i32)
        self.offsets = torch.empty((E + 1,), **i32)
        self.sorted_slot = torch.empty((T * k,), **i32)
        self.slot_pos = torch.empty((T * k,), **i32)
        self.max_blocks = moe_max_blocks(d)
        if self.max_blocks < 0:
            raise MoeError(MOE_EINVAL, "moe_max_blocks")
        self.blocks = torch.empty((max(self.max_blocks, 1), 4), **i32)
        self.n_blocks = torch.empty((1,), **i32)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=device) if export_logits else None
        self.status = torch.zeros((1,), **i32)
        self.ws_bytes = moe_route_ws_bytes(d)
        self.ws = torch.empty((max(self.ws_bytes, 16),), dtype=torch.uint8, device=device)
        self.c = RouteOut(self.topk_idx.data_ptr(), self.topk_w.data_ptr(), self.counts.data_ptr(),
                          self.offsets.data_ptr(), self.sorted_slot.data_ptr(),
                          self.slot_pos.data_ptr(), self.blocks.data_ptr(),
                          self.n_blocks.data_ptr(),
                          self.logits.data_ptr() if self.logits is not None else None,
                          self.status.data_ptr(), self.ws.data_ptr(), self.ws_bytes)

    def host(self) -> dict:
        """Copy every table to host numpy arrays (synchronising)."""
        nb = int(self.n_blocks.item())
        out = dict(topk_idx=self.topk_idx.cpu().numpy(), topk_w=self.topk_w.cpu().numpy(),
                   counts=self.counts.cpu().numpy(), offsets=self.offsets.cpu().numpy(),
                   sorted_slot=self.sorted_slot.cpu().numpy(), slot_pos=self.slot_pos.cpu().numpy(),
                   blocks=self.blocks[:nb].cpu().numpy(), n_blocks=nb,
                   status=int(self.status.item()) & 0xFFFFFFFF)
        if self.logits is not None:
            out["logits"] = self.logits.cpu().numpy()
        return out


class MoeLayer:
    """One MoE layer resident on the device: weights, router and work buffers.

    forward(x) enqueues moe_route, moe_w4_gate_up, moe_w4_down and moe_combine
    on the current stream; nothing synchronises.
    """

    def __init__(self, H, I, E, k, n_shared, routed: DeviceBank, shared, w_router, logit_bias=None,
                 T_max=2048, tile_m_max=128, tile_gran=16, device="cuda", export_logits=False):
        import torch
        self.H, self.I, self.E, self.k, self.n_shared = H, I, E, k, n_shared
        self.routed, self.shared = routed, shared
        self.w_router = w_router if not isinstance(w_router, np.ndarray) else _dev(w_router, device)
        self.bias = (None if logit_bias is None else
                     logit_bias if not isinstance(logit_bias, np.ndarray) else _dev(logit_bias, device))
        self.tile_m_max, self.tile_gran = tile_m_max, tile_gran
        self.T_max = T_max
        self.dmax = make_dims(T_max, H, I, E, k, n_shared, tile_m_max, tile_gran)
        self.rt = RouteTables(self.dmax, device, export_logits)
        rows = T_max * k + (T_max if n_shared else 0)
        self.h = torch.empty((rows, I), dtype=torch.int16, device=device)
        self.y_slots = torch.empty((rows, H), dtype=torch.int16, device=device)
        # forward_residual's normed rows: the router and gate/up have read them before down writes y_slots
        self.xn = self.y_slots[:T_max]

    def dims(self, T):
        if T > self.T_max:
            raise ValueError(f"T={T} exceeds the layer's T_max={self.T_max}")
        return make_dims(T, self.H, self.I, self.E, self.k, self.n_shared, self.tile_m_max,
                         self.tile_gran)

    def route(self, x, T=None, stream=None):
        d = self.dims(x.shape[0] if T is None else T)
        moe_route(d, x, self.w_router, self.bias, self.rt.c, stream)
        return d

    def gate_up(self, d, x, routed=None, shared=None, stream=None):
        r = routed or self.routed
        s = shared or self.shared
        moe_w4_gate_up(d, x, self.rt.c, r.c, s.c if s is not None else None, self.h, stream)

    def down(self, d, routed=None, shared=None, stream=None):
        r = routed or self.routed
        s = shared or self.shared
        moe_w4_down(d, self.rt.c, r.c, s.c if s is not None else None, self.h, self.y_slots, stream)

    def ffn(self, d, x, routed=None, shared=None, stream=None):
        """gate/up then down through the library's grouped call."""
        r = routed or self.routed
        s = shared or self.shared
        moe_grouped_w4_ffn(d, x, self.rt.c, r.c, s.c if s is not None else None, self.h,
                           self.y_slots, stream)

    def shared_ffn(self, d, x, shared=None, stream=None):
        """The shared expert's rows of h and y_slots; needs no routing."""
        s = shared or self.shared
        moe_shared_w4_ffn(d, x, s.c, self.h, self.y_slots, stream)

    def routed_ffn(self, d, x, routed=None, stream=None):
        """The routed rows of h and y_slots (after route on the same stream)."""
        r = routed or self.routed
        moe_routed_w4_ffn(d, x, self.rt.c, r.c, self.h, self.y_slots, stream)

    def combine(self, d, y, stream=None):
        moe_combine(d, self.rt.c, self.y_slots, y, stream)

    def ffn_combine(self, d, x, y, routed=None, shared=None, stream=None):
        """gate/up, down and combine in one library call (down and combine
        fused for a single token)."""
        r = routed or self.routed
        s = shared or self.shared
        moe_w4_ffn_combine(d, x, self.rt.c, r.c, s.c if s is not None else None, self.h,
                           self.y_slots, y, stream)

    def forward(self, x, y, routed=None, shared=None, stream=None):
        d = self.route(x, stream=stream)
        self.ffn_combine(d, x, y, routed, shared, stream)
        return y

    def _residual_dims(self, x, y):
        """Sizes of a forward_residual call; y is checked before res is added to."""
        d = self.dims(x.shape[0])
        _arg(y, 2 * d.T * self.H, "y", _device(), _BF16)
        return d

    def forward_residual(self, x, res, norm_weight, y, eps=1e-6, stream=None):
        """The layer with what stands in front of it: res += x in place, then
        the layer on the RMS norm of the sum (bfloat16 rows of at most NORM_MAX_H
        elements, one norm call)."""
        d = self._residual_dims(x, y)
        moe_add_rmsnorm(NormDims(d.T, self.H, ELEM_BF16, eps), x, res, norm_weight, res, self.xn,
                        stream=stream)
        return self.forward(self.xn[:d.T], y, stream=stream)


class Q8MoeLayer(MoeLayer):
    """The same layer with 8-bit banks (DeviceBankQ8): routing and combine as in
    MoeLayer, the products in 8-bit integers.  gate_up, and so forward, quantises
    the tokens itself; forward_residual gets them from the norm.  H and I are at
    most NORM_MAX_H.  A bank of other sizes than the layer's, or with fewer
    experts, is refused."""

    def __init__(self, H, I, *args, device="cuda", **kw):
        import torch
        _check_q8_widths(H, I)
        super().__init__(H, I, *args, device=device, **kw)
        self._banks()
        rows = self.h.shape[0]
        self.xn = torch.empty((self.T_max, H), dtype=torch.int16, device=device)   # kept next to their 8-bit form
        self.xq = torch.empty((self.T_max, self.H), dtype=torch.int8, device=device)
        self.xs = torch.empty((self.T_max,), dtype=torch.float32, device=device)
        self.hq = torch.empty((rows, self.I), dtype=torch.int8, device=device)
        self.hs = torch.empty((rows,), dtype=torch.float32, device=device)

    def gate_up(self, d, x, routed=None, shared=None, stream=None):
        self._gate_up(d, self._banks(routed, shared), x, stream)

    def down(self, d, routed=None, shared=None, stream=None):
        self._down(d, self._banks(routed, shared), stream)

    def ffn(self, d, x, routed=None, shared=None, stream=None):
        banks = self._banks(routed, shared)
        self._gate_up(d, banks, x, stream)
        self._down(d, banks, stream)

    def _banks(self, routed=None, shared=None):
        """The C structs of the banks of a call (None: the layer's own); the kernels read them by the
        layer's sizes."""
        routed, shared = routed or self.routed, (shared or self.shared) if self.n_shared else None
        for what, bank, n in (("routed", routed, self.E), ("shared", shared, 1)):
            if bank is not None and not (isinstance(bank, DeviceBankQ8) and bank.n >= n and bank.H == self.H and
                                         bank.I == self.I and bank.t["gu"].get_device() == self.h.get_device()):
                raise ValueError(f"{what}: a DeviceBankQ8 of {n} experts, H {self.H}, I {self.I} on {self.h.device} "
                                 f"is needed, got {bank}")
        return None if routed is None else routed.c, None if shared is None else shared.c

    def _gate_up(self, d, banks, x, stream):
        moe_q8_quantize(NormDims(d.T, self.H, ELEM_BF16, 0.0), x, self.xq, self.xs, stream)
        moe_q8_gate_up(d, self.xq, self.xs, self.rt.c, *banks, self.h, stream)

    def _down(self, d, banks, stream):
        rows = _rows_of(d)
        moe_q8_quantize(NormDims(min(rows, NORM_MAX_T), self.I, ELEM_BF16, 0.0), self.h, self.hq, self.hs, stream)
        for lo in range(NORM_MAX_T, rows, NORM_MAX_T):   # up to 33 * 2^20 rows
            moe_q8_quantize(NormDims(min(rows - lo, NORM_MAX_T), self.I, ELEM_BF16, 0.0), self.h[lo:], self.hq[lo:],
                            self.hs[lo:], stream)
        moe_q8_down(d, self.rt.c, *banks, self.hq, self.hs, self.y_slots, stream)

    def shared_ffn(self, d, x, shared=None, stream=None):
        raise NotImplementedError("the 8-bit layer has no split of the shared expert")

    routed_ffn = shared_ffn

    def ffn_combine(self, d, x, y, routed=None, shared=None, stream=None):
        self.ffn(d, x, routed, shared, stream)
        self.combine(d, y, stream)

    def forward_residual(self, x, res, norm_weight, y, eps=1e-6, stream=None):
        d, banks = self._residual_dims(x, y), self._banks()
        moe_add_rmsnorm(NormDims(d.T, self.H, ELEM_BF16, eps), x, res, norm_weight, res, self.xn,
                        self.xq, self.xs, stream)
        self.route(self.xn[:d.T], stream=stream)
        moe_q8_gate_up(d, self.xq, self.xs, self.rt.c, *banks, self.h, stream)
        self._down(d, banks, stream)
        self.combine(d, y, stream)
        return y
