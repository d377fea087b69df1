"""Thin ctypes binding of libdmoe.so (declared in include/dmoe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels.
PyTorch is used for device memory and streams.  There is no fallback: if the library is
missing or the device is not a B200 the calls raise.

The functions carry the C names (``dmoe_sparse_map``, ``dmoe_forward``, ``dmoe_backward`` and
the step entry points) and take torch tensors where the C call takes device pointers.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from .build import LIB

BLOCKING = 128
MAX_EXPERTS = 1024
MAX_TOP_K = 32

FEW_MAX_TOKENS = 128

WS_MAP, WS_FORWARD, WS_BACKWARD, WS_FORWARD_TRAIN, WS_ROUTER_BACKWARD = 0, 1, 2, 3, 4
WS_FEW, WS_MX4_FORWARD = 6, 7
DGLU_TILE_COLS = 128

STATUS_NONFINITE_LOGITS = 0x1
STATUS_EXPERT_OUT_OF_RANGE = 0x2
STATUS_DUPLICATE_EXPERT = 0x4
STATUS_TIMEOUT = 0x8

_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_I = ctypes.c_int


ROUTE_RENORMALIZE = 0x1
ROUTE_TOKEN_ROUNDING = 0x2
SAVE_X_ONLY = 0x4
FUSED_COMBINE = 0x8
SCALE_COLS = 128  # block floating point of Y_pad / dX_pad: one scale per row and 128 columns


def scale_stride(h: int) -> int:
    """Row stride of the scale arrays: ceil(h/128) scales padded to a multiple of 4."""
    return (h + 511) // 512 * 4


class dmoe_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("flags", ctypes.c_int32)]

    def __repr__(self):
        return (f"dmoe_dims(T={self.T}, hidden={self.hidden}, ffn={self.ffn}, "
                f"num_experts={self.num_experts}, top_k={self.top_k}, "
                f"flags={self.flags})")


MAP_FIELDS = ("top_experts", "weights", "tokens_per_expert", "bins", "padded_bins", "indices",
              "bin_ids", "dest_row", "block_expert", "num_blocks", "status", "entry_offsets")


class dmoe_map(ctypes.Structure):
    _fields_ = [(n, _P) for n in MAP_FIELDS]


class dmoe_mx4(ctypes.Structure):
    _fields_ = [("codes", _P), ("scales", _P)]


class DMoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {error_string(code)} ({code})")
        self.code = code


_lib = None


def load():
    """Load the in-tree libdmoe.so (build it first with ``build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise ImportError(f"libdmoe.so not built: {LIB} is missing "
                          "(run python -m dropless_mixture_experts_dmoe_b200.build)")
    lib = ctypes.CDLL(LIB)
    D = ctypes.POINTER(dmoe_dims)
    M = ctypes.POINTER(dmoe_map)
    lib.dmoe_padded_rows_max.argtypes = [D]
    lib.dmoe_padded_rows_max.restype = _SZ
    lib.dmoe_entries_max.argtypes = [D]
    lib.dmoe_entries_max.restype = _SZ
    lib.dmoe_workspace_bytes.argtypes = [D, _I]
    lib.dmoe_workspace_bytes.restype = _SZ
    lib.dmoe_saved_bytes.argtypes = [D, ctypes.POINTER(_SZ)]
    lib.dmoe_saved_bytes.restype = _SZ
    lib.dmoe_sparse_map.argtypes = [D, _P, M, _P, _SZ, _P]
    lib.dmoe_forward.argtypes = [D, _P, _P, _P, _P, M, _P, _P, _P, _SZ, _P]
    lib.dmoe_backward.argtypes = [D, _P, _P, _P, _P, M, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
    lib.dmoe_padded_gather.argtypes = [D, _P, M, _P, _P]
    lib.dmoe_expert_glu.argtypes = [D, _P, _P, _P, M, _P, _P, _P, _P]
    lib.dmoe_expert_glu_gather.argtypes = [D, _P, _P, _P, M, _P, _P, _P, _P]
    lib.dmoe_expert_down.argtypes = [D, _P, _P, M, _P, _P, _P]
    lib.dmoe_padded_scatter.argtypes = [D, _P, _P, M, _P, _P, _P]
    lib.dmoe_expert_down_combine.argtypes = [D, _P, _P, M, _P, _P, _P]
    lib.dmoe_bwd_dglu.argtypes = [D, _P, _P, _P, _P, M, _P, _P, _P, _P, _P]
    lib.dmoe_bwd_scatter.argtypes = [D, _P, _P, _P, M, _P, _P, _P]
    lib.dmoe_router_forward.argtypes = [D, _P, _P, _P, _P, _P]
    lib.dmoe_router_dlogits.argtypes = [D, _P, M, _P, _P, _P]
    lib.dmoe_router_backward.argtypes = [D, _P, _P, _P, M, _P, _P, _P, _P, _SZ, _P]
    lib.dmoe_bwd_dx.argtypes = [D, _P, _P, _P, _P, M, _P, _P, _P]
    lib.dmoe_bwd_wgrad.argtypes = [D, _P, _P, _P, _P, _P, M, _P, _P, _P, _P]
    lib.dmoe_sparse_map_noalloc.argtypes = [D, _P, M, _P]
    Q = ctypes.POINTER(dmoe_mx4)
    i64 = ctypes.c_int64
    lib.dmoe_forward_few.argtypes = [D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
    lib.dmoe_mx4_forward_few.argtypes = [D, _P, _P, Q, Q, Q, _P, _P, _P, _P, _P, _SZ, _P]
    lib.dmoe_mx4_quantize.argtypes = [i64, i64, _P, Q, _P]
    lib.dmoe_mx4_dequantize.argtypes = [i64, i64, Q, _P, _P]
    lib.dmoe_mx4_forward.argtypes = [D, _P, Q, Q, Q, M, _P, _P, _SZ, _P]
    for fn in ("dmoe_sparse_map", "dmoe_sparse_map_noalloc", "dmoe_forward", "dmoe_backward",
               "dmoe_padded_gather",
               "dmoe_expert_glu", "dmoe_expert_glu_gather", "dmoe_expert_down", "dmoe_padded_scatter",
               "dmoe_expert_down_combine",
               "dmoe_bwd_dglu", "dmoe_bwd_dx", "dmoe_bwd_wgrad", "dmoe_bwd_scatter",
               "dmoe_router_forward", "dmoe_router_dlogits", "dmoe_router_backward",
               "dmoe_forward_few", "dmoe_mx4_forward_few", "dmoe_mx4_quantize",
               "dmoe_mx4_dequantize", "dmoe_mx4_forward"):
        getattr(lib, fn).restype = _I
    lib.dmoe_error_string.argtypes = [_I]
    lib.dmoe_error_string.restype = ctypes.c_char_p
    lib.dmoe_status_string.argtypes = [ctypes.c_int32]
    lib.dmoe_status_string.restype = ctypes.c_char_p
    lib.dmoe_version.argtypes = []
    lib.dmoe_version.restype = ctypes.c_char_p
    lib.dmoe_debug_inject_stall.argtypes = [_I]
    lib.dmoe_debug_inject_stall.restype = _I
    _lib = lib
    return lib


def error_string(code: int) -> str:
    return load().dmoe_error_string(code).decode()


def status_string(status: int) -> str:
    return load().dmoe_status_string(int(status)).decode()


def version() -> str:
    return load().dmoe_version().decode()


def dmoe_debug_inject_stall(nth: int = 1) -> None:
    """Test-only: the nth product-kernel launch from now (True: the next; 0: none) stalls on
    purpose and reports STATUS_TIMEOUT (see include/dmoe.h)."""
    _check(load().dmoe_debug_inject_stall(int(nth)), "dmoe_debug_inject_stall")


def make_dims(T: int, hidden: int, ffn: int, num_experts: int, top_k: int,
              flags: int = 0) -> dmoe_dims:
    """flags: an OR of ROUTE_RENORMALIZE (weights = softmax over the k chosen logits) and
    SAVE_X_ONLY (the forward saves X_pad only; the backward recomputes A and Bm)."""
    return dmoe_dims(T, hidden, ffn, num_experts, top_k, flags)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the raw handle: a torch Stream object costs three microseconds more
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str):
    if rc != 0:
        raise DMoEError(rc, what)


# ---- sizes ------------------------------------------------------------------------------------

def dmoe_padded_rows_max(dims: dmoe_dims) -> int:
    return int(load().dmoe_padded_rows_max(ctypes.byref(dims)))


def dmoe_entries_max(dims: dmoe_dims) -> int:
    return int(load().dmoe_entries_max(ctypes.byref(dims)))


def dmoe_workspace_bytes(dims: dmoe_dims, kind: int) -> int:
    return int(load().dmoe_workspace_bytes(ctypes.byref(dims), kind))


def dmoe_saved_bytes(dims: dmoe_dims):
    offs = (_SZ * 3)()
    total = int(load().dmoe_saved_bytes(ctypes.byref(dims), offs))
    return total, [int(o) for o in offs]


# ---- the sparse map -----------------------------------------------------------------------------

class SparseMap:
    """Device tensors of the sparse map (torch allocations) and their C view."""

    def __init__(self, dims: dmoe_dims, device="cuda"):
        T, E, k = dims.T, dims.num_experts, dims.top_k
        P = dmoe_padded_rows_max(dims)
        if P == 0:
            raise DMoEError(-2, "SparseMap")
        i32 = dict(dtype=torch.int32, device=device)
        self.dims = dims
        self._kind = _map_kind(dims)  # dims is the caller's object, which may change
        rounding = bool(dims.flags & ROUTE_TOKEN_ROUNDING)
        N = dmoe_entries_max(dims)
        if rounding:  # experts and weights of the token-major entry list
            self.top_experts = torch.empty(N, **i32)
            self.weights = torch.empty(N, dtype=torch.float32, device=device)
        else:
            self.top_experts = torch.empty((T, k), **i32)
            self.weights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.tokens_per_expert = torch.empty(E, **i32)
        self.bins = torch.empty(E, **i32)
        self.padded_bins = torch.empty(E, **i32)
        self.indices = torch.empty(N, **i32)
        self.bin_ids = torch.empty(N, **i32)
        self.dest_row = torch.empty(N, **i32)
        self.block_expert = torch.empty(max(P // BLOCKING, 1), **i32)
        self.num_blocks = torch.empty(1, **i32)
        self.status = torch.zeros(1, **i32)
        # token rounding: a token-major entry list (see include/dmoe.h)
        self.entry_offsets = torch.empty(T + 1, **i32) if rounding else None
        self._c = dmoe_map(*[0 if getattr(self, n) is None else getattr(self, n).data_ptr()
                             for n in MAP_FIELDS])

    @property
    def c(self) -> dmoe_map:
        return self._c

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n in MAP_FIELDS if getattr(self, n) is not None}


def dmoe_sparse_map(dims: dmoe_dims, logits, smap: SparseMap, ws, stream=None):
    """Routing + sparse map.  logits: [T,E] bf16 CUDA tensor or None (top_experts given)."""
    ws_bytes = ws.numel() * ws.element_size()
    rc = load().dmoe_sparse_map(ctypes.byref(dims), _ptr(logits), ctypes.byref(smap.c), _ptr(ws),
                                ws_bytes, _stream(stream))
    _check(rc, "dmoe_sparse_map")


def dmoe_forward(dims: dmoe_dims, x, w1, w3, w2, smap: SparseMap, y, saved=None, ws=None,
                 stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().dmoe_forward(ctypes.byref(dims), _ptr(x), _ptr(w1), _ptr(w3), _ptr(w2),
                             ctypes.byref(smap.c), _ptr(y), _ptr(saved), _ptr(ws), ws_bytes,
                             _stream(stream))
    _check(rc, "dmoe_forward")


def dmoe_backward(dims: dmoe_dims, dy, w1, w3, w2, smap: SparseMap, saved, dx, dw1, dw3, dw2,
                  dweights, ws, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().dmoe_backward(ctypes.byref(dims), _ptr(dy), _ptr(w1), _ptr(w3), _ptr(w2),
                              ctypes.byref(smap.c), _ptr(saved), _ptr(dx), _ptr(dw1), _ptr(dw3),
                              _ptr(dw2), _ptr(dweights), _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "dmoe_backward")


def dmoe_padded_gather(dims, x, smap: SparseMap, x_pad, stream=None):
    _check(load().dmoe_padded_gather(ctypes.byref(dims), _ptr(x), ctypes.byref(smap.c), _ptr(x_pad),
                                     _stream(stream)), "dmoe_padded_gather")


def dmoe_expert_glu(dims, x_pad, w1, w3, smap: SparseMap, h_out, a_out=None, b_out=None,
                    stream=None):
    _check(load().dmoe_expert_glu(ctypes.byref(dims), _ptr(x_pad), _ptr(w1), _ptr(w3),
                                  ctypes.byref(smap.c), _ptr(h_out), _ptr(a_out), _ptr(b_out),
                                  _stream(stream)), "dmoe_expert_glu")


def dmoe_expert_glu_gather(dims, x, w1, w3, smap: SparseMap, h_out, a_out=None, b_out=None,
                           stream=None):
    _check(load().dmoe_expert_glu_gather(ctypes.byref(dims), _ptr(x), _ptr(w1), _ptr(w3),
                                         ctypes.byref(smap.c), _ptr(h_out), _ptr(a_out),
                                         _ptr(b_out), _stream(stream)), "dmoe_expert_glu_gather")


def dmoe_expert_down(dims, h_in, w2, smap: SparseMap, y_pad, y_scale, stream=None):
    """y_pad [P_max,h] fp16 and y_scale [P_max, scale_stride(h)] fp32: block floating point."""
    _check(load().dmoe_expert_down(ctypes.byref(dims), _ptr(h_in), _ptr(w2), ctypes.byref(smap.c),
                                   _ptr(y_pad), _ptr(y_scale), _stream(stream)), "dmoe_expert_down")


def dmoe_expert_down_combine(dims, h_in, w2, smap: SparseMap, y, y_acc, stream=None):
    """y = the weighted combine of the down GEMM, fused (y_acc: T*h fp32 workspace)."""
    _check(load().dmoe_expert_down_combine(ctypes.byref(dims), _ptr(h_in), _ptr(w2),
                                           ctypes.byref(smap.c), _ptr(y), _ptr(y_acc),
                                           _stream(stream)), "dmoe_expert_down_combine")


def dmoe_padded_scatter(dims, y_pad, y_scale, smap: SparseMap, weights, y, stream=None):
    """y_scale None: y_pad is bf16; else block floating point (fp16 y_pad and its scales)."""
    _check(load().dmoe_padded_scatter(ctypes.byref(dims), _ptr(y_pad), _ptr(y_scale),
                                      ctypes.byref(smap.c), _ptr(weights), _ptr(y),
                                      _stream(stream)), "dmoe_padded_scatter")


def dmoe_bwd_dglu(dims, dy_pad, w2, a_saved, bm_saved, smap: SparseMap, da, dbm, hw, dw_part,
                  stream=None):
    _check(load().dmoe_bwd_dglu(ctypes.byref(dims), _ptr(dy_pad), _ptr(w2), _ptr(a_saved),
                                _ptr(bm_saved), ctypes.byref(smap.c), _ptr(da), _ptr(dbm),
                                _ptr(hw), _ptr(dw_part), _stream(stream)), "dmoe_bwd_dglu")


def dmoe_bwd_scatter(dims, dx_pad, dx_scale, dw_part, smap: SparseMap, dx, dweights,
                     stream=None):
    _check(load().dmoe_bwd_scatter(ctypes.byref(dims), _ptr(dx_pad), _ptr(dx_scale),
                                   _ptr(dw_part), ctypes.byref(smap.c), _ptr(dx), _ptr(dweights),
                                   _stream(stream)), "dmoe_bwd_scatter")


def dmoe_bwd_dx(dims, da, dbm, w1, w3, smap: SparseMap, dx_pad, dx_scale, stream=None):
    """dx_pad [P_max,h] fp16 and dx_scale [P_max, scale_stride(h)] fp32: block floating point."""
    _check(load().dmoe_bwd_dx(ctypes.byref(dims), _ptr(da), _ptr(dbm), _ptr(w1), _ptr(w3),
                              ctypes.byref(smap.c), _ptr(dx_pad), _ptr(dx_scale),
                              _stream(stream)), "dmoe_bwd_dx")


def dmoe_bwd_wgrad(dims, x_pad, hw, dy_pad, da, dbm, smap: SparseMap, dw1, dw3, dw2,
                   stream=None):
    _check(load().dmoe_bwd_wgrad(ctypes.byref(dims), _ptr(x_pad), _ptr(hw), _ptr(dy_pad),
                                 _ptr(da), _ptr(dbm), ctypes.byref(smap.c), _ptr(dw1), _ptr(dw3),
                                 _ptr(dw2), _stream(stream)), "dmoe_bwd_wgrad")


def dmoe_router_forward(dims, x, w_router, logits, status, stream=None):
    """logits [T,E] bf16 = x W_r^T (the linear router; E % 8 == 0)."""
    _check(load().dmoe_router_forward(ctypes.byref(dims), _ptr(x), _ptr(w_router), _ptr(logits),
                                      _ptr(status), _stream(stream)), "dmoe_router_forward")


def dmoe_router_dlogits(dims, logits, smap: SparseMap, dweights, dlogits, stream=None):
    _check(load().dmoe_router_dlogits(ctypes.byref(dims), _ptr(logits), ctypes.byref(smap.c),
                                      _ptr(dweights), _ptr(dlogits), _stream(stream)),
           "dmoe_router_dlogits")


def dmoe_router_backward(dims, x, w_router, logits, smap: SparseMap, dweights, dx, dw_router, ws,
                         stream=None):
    """dx += dlogits W_r (in place), dw_router = dlogits^T x (fp32)."""
    ws_bytes = ws.numel() * ws.element_size()
    _check(load().dmoe_router_backward(ctypes.byref(dims), _ptr(x), _ptr(w_router), _ptr(logits),
                                       ctypes.byref(smap.c), _ptr(dweights), _ptr(dx),
                                       _ptr(dw_router), _ptr(ws), ws_bytes, _stream(stream)),
           "dmoe_router_backward")


def dmoe_sparse_map_noalloc(dims: dmoe_dims, logits, smap: SparseMap, stream=None):
    """Allocation-free routing + sparse map (static scratch inside the library; see
    include/dmoe.h).  For callers that cannot allocate a workspace."""
    _check(load().dmoe_sparse_map_noalloc(ctypes.byref(dims), _ptr(logits),
                                          ctypes.byref(smap.c), _stream(stream)),
           "dmoe_sparse_map_noalloc")


# ---- serving: the layer for a few tokens, and the microscaled 4-bit format ------------------------

def _device() -> int:
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2


def _stream_on(device: int, stream) -> int | None:
    """_stream for callers that have the current device."""
    return (torch._C._cuda_getCurrentRawStream(device) if stream is None and device >= 0 else
            _stream(stream))


def _arg(name: str, t, shape: tuple, dtype, device: int) -> int:
    """Address of an argument of the serving calls: a contiguous tensor of this shape and type on
    the current CUDA device (a raw device address is passed on as it is)."""
    if isinstance(t, int):
        return t
    if (t.get_device() != device or t.dtype != dtype or t.shape != shape or
            not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"the current CUDA device; got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class Mx4:
    """A matrix, or a stack of expert matrices, in the microscaled 4-bit format (see dmoe_mx4 in
    include/dmoe.h): ``codes`` [..., rows, cols / 2] and ``scales`` [..., ceil(rows/128), cols/128,
    32, 4, 4], contiguous uint8 tensors, fixed for the object's life.  In a stack ``rows`` is a
    multiple of 128."""

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not (
                codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous uint8 tensors")
        self.shape = (*codes.shape[:-1], 2 * codes.shape[-1])
        if codes.dim() < 2 or tuple(scales.shape) != self.scales_shape(*self.shape):
            raise ValueError(f"scales of codes {tuple(codes.shape)}: {tuple(scales.shape)}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self._codes, self._scales = codes, scales
        self._device = codes.get_device()
        self._size = (math.prod(self.shape[:-1]), self.shape[-1])
        self._c = dmoe_mx4(codes.data_ptr(), scales.data_ptr())
        self.ref = ctypes.byref(self._c)

    def arg(self, name: str, shape: tuple, device: int):
        """This matrix as an argument: of this shape, on the current CUDA device."""
        if self.shape != shape or self._device != device:
            raise ValueError(f"{name} must have shape {shape} on the current CUDA device; got "
                             f"{self.shape} on {self.codes.device}")
        return self.ref

    @staticmethod
    def scales_shape(*shape) -> tuple:
        """Shape of the scale tensor of a [..., rows, cols] matrix."""
        *lead, rows, cols = shape
        if rows < 1 or cols < 128 or cols % 128 or (lead and rows % 128):
            raise ValueError("cols, and the rows of a stack, must be multiples of 128")
        return (*lead, (rows + 127) // 128, cols // 128, 32, 4, 4)

    @classmethod
    def empty(cls, *shape, device="cuda") -> "Mx4":
        scales = cls.scales_shape(*shape)
        return cls(torch.empty((*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device=device),
                   torch.empty(scales, dtype=torch.uint8, device=device))


def dmoe_mx4_quantize(src, dst: Mx4, stream=None):
    """dst = src (bf16, the shape of dst) in the microscaled 4-bit format."""
    rows, cols = dst._size
    dev = _device()
    _check(load().dmoe_mx4_quantize(rows, cols, _arg("src", src, dst.shape, torch.bfloat16, dev),
                                    dst.arg("dst", dst.shape, dev), _stream_on(dev, stream)),
           "dmoe_mx4_quantize")


def dmoe_mx4_dequantize(src: Mx4, dst, stream=None):
    """dst (bf16) = the values of src."""
    rows, cols = src._size
    dev = _device()
    _check(load().dmoe_mx4_dequantize(rows, cols, src.arg("src", src.shape, dev),
                                      _arg("dst", dst, src.shape, torch.bfloat16, dev),
                                      _stream_on(dev, stream)), "dmoe_mx4_dequantize")


class FewBuffers:
    """Device buffers of the few-token calls for one shape: ``top_experts`` [T,k] and ``weights``
    [T,k] (outputs when logits are given, else inputs: copy the given routing into them),
    ``status`` (starts at 0, bits are OR-ed in) and the workspace ``ws``."""

    top_experts = property(lambda self: self._tensors[0])
    weights = property(lambda self: self._tensors[1])
    status = property(lambda self: self._tensors[2])
    ws = property(lambda self: self._tensors[3])

    def __init__(self, dims: dmoe_dims, device="cuda"):
        n = dmoe_workspace_bytes(dims, WS_FEW)
        if n == 0:
            raise DMoEError(-2, "FewBuffers")
        self.dims = dims
        self._sizes = _sizes(dims)
        self._tensors = (
            torch.empty((dims.T, dims.top_k), dtype=torch.int32, device=device),
            torch.empty((dims.T, dims.top_k), dtype=torch.float32, device=device),
            torch.zeros(1, dtype=torch.int32, device=device),
            torch.empty(n, dtype=torch.uint8, device=device))
        self._device = self.ws.get_device()
        self._args = (*(t.data_ptr() for t in self._tensors), n)

    def args(self, device: int) -> tuple:
        """Addresses of the buffers and the size of ws, on the current CUDA device."""
        if self._device != device:
            raise ValueError("the buffers must be on the current CUDA device; they are on "
                             f"{self.ws.device}")
        return self._args


def _sizes(dims) -> tuple:
    return dims.T, dims.hidden, dims.ffn, dims.num_experts, dims.top_k


def _map_kind(dims) -> tuple:
    """What a map is made for: the sizes, and whether it is token rounding's entry list."""
    return (*_sizes(dims), bool(dims.flags & ROUTE_TOKEN_ROUNDING))


def _few_args(dims, x, logits, bufs, y, dev):
    if bufs._sizes != _sizes(dims):
        raise ValueError(f"the buffers are those of sizes {bufs._sizes}, not of {_sizes(dims)}")
    row = (dims.T, dims.hidden)
    return (_arg("x", x, row, torch.bfloat16, dev),
            None if logits is None else _arg("logits", logits, (dims.T, dims.num_experts),
                                             torch.bfloat16, dev),
            _arg("y", y, row, torch.bfloat16, dev))


def dmoe_forward_few(dims: dmoe_dims, x, logits, w1, w3, w2, bufs: FewBuffers, y, stream=None):
    """The whole layer for T <= FEW_MAX_TOKENS tokens, from the logits [T,E] to y [T,h].  logits
    None: bufs.top_experts and bufs.weights are taken as given."""
    dev = _device()
    xp, lp, yp = _few_args(dims, x, logits, bufs, y, dev)
    E, h, f, bf = dims.num_experts, dims.hidden, dims.ffn, torch.bfloat16
    w = (_arg("w1", w1, (E, f, h), bf, dev), _arg("w3", w3, (E, f, h), bf, dev),
         _arg("w2", w2, (E, h, f), bf, dev))
    top, weights, status, ws, n = bufs.args(dev)
    _check(load().dmoe_forward_few(ctypes.byref(dims), xp, lp, *w, top, weights, yp, status, ws, n,
                                   _stream_on(dev, stream)), "dmoe_forward_few")


def dmoe_mx4_forward_few(dims: dmoe_dims, x, logits, w1: Mx4, w3: Mx4, w2: Mx4, bufs: FewBuffers,
                         y, stream=None):
    """dmoe_forward_few over expert weights in the microscaled 4-bit format."""
    dev = _device()
    xp, lp, yp = _few_args(dims, x, logits, bufs, y, dev)
    E, h, f = dims.num_experts, dims.hidden, dims.ffn
    w = (w1.arg("w1", (E, f, h), dev), w3.arg("w3", (E, f, h), dev), w2.arg("w2", (E, h, f), dev))
    top, weights, status, ws, n = bufs.args(dev)
    _check(load().dmoe_mx4_forward_few(ctypes.byref(dims), xp, lp, *w, top, weights, yp, status,
                                       ws, n, _stream_on(dev, stream)), "dmoe_mx4_forward_few")


class Mx4Buffers:
    """Device buffers of the 4-bit layer over many tokens for one shape: the sparse map and its
    workspace, and the forward's workspace ``ws``.  After a forward ``hidden()`` is a view of the
    workspace: H of the padded rows in the 4-bit format."""

    def __init__(self, dims: dmoe_dims, device="cuda"):
        self.dims = dims
        self.map = SparseMap(dims, device)
        u8 = dict(dtype=torch.uint8, device=device)
        self.ws_map = torch.empty(max(dmoe_workspace_bytes(dims, WS_MAP), 16), **u8)
        self.ws = torch.empty(dmoe_workspace_bytes(dims, WS_MX4_FORWARD), **u8)

    def hidden(self) -> Mx4:
        P, h, f = dmoe_padded_rows_max(self.dims), self.dims.hidden, self.dims.ffn
        up = lambda v: (v + 255) // 256 * 256
        o_q = up(up(P * h // 2) + P * h // 32)
        o_s = up(o_q + P * f // 2)
        return Mx4(self.ws[o_q:o_q + P * f // 2].view(P, f // 2),
                   self.ws[o_s:o_s + P * f // 32].view(Mx4.scales_shape(P, f)))


def dmoe_mx4_forward(dims: dmoe_dims, x, w1: Mx4, w3: Mx4, w2: Mx4, smap: SparseMap, y, ws,
                     stream=None):
    """y [T,h] = the layer with every product in the microscaled 4-bit format (inference)."""
    E, h, f, row = dims.num_experts, dims.hidden, dims.ffn, (dims.T, dims.hidden)
    dev = _device()
    if smap._kind != _map_kind(dims):
        raise ValueError("the map is that of (T, hidden, ffn, num_experts, top_k, token rounding) = "
                         f"{smap._kind}, not of {_map_kind(dims)}")
    _arg("smap.status", smap.status, (1,), torch.int32, dev)
    _check(load().dmoe_mx4_forward(ctypes.byref(dims), _arg("x", x, row, torch.bfloat16, dev),
                                   w1.arg("w1", (E, f, h), dev), w3.arg("w3", (E, f, h), dev),
                                   w2.arg("w2", (E, h, f), dev), ctypes.byref(smap.c),
                                   _arg("y", y, row, torch.bfloat16, dev),
                                   _arg("ws", ws, ws.shape, ws.dtype, dev),
                                   ws.numel() * ws.element_size(), _stream_on(dev, stream)),
           "dmoe_mx4_forward")


# ---- buffers (allocation only) ----------------------------------------------------------------

class Buffers:
    """Caller-side device allocations for one layer shape: map, workspaces, saved activations.

    train=True: ``saved`` (X_pad, A, Bm for the backward), the training forward workspace
    ``ws_fwd`` (H, Y_pad and its scales), the backward workspace, and separate step buffers
    ``bstep`` (dy_pad, da, dbm, hw, dw_part, dx_pad, dx_scale) for driving the backward step
    entry points one by one.  train=False: the inference workspace of ``dmoe_forward`` plus
    separate X_pad / H / Y_pad / Y_pad-scale tensors (``step``) for the forward step entry
    points.  ``view(name)`` gives [P_max, cols] views: x_pad, a, bm (bf16) of the saved buffer,
    and h (bf16), y_pad (fp16) and y_scale (fp32) of the forward workspace (valid until the
    workspace is reused)."""

    def __init__(self, dims: dmoe_dims, train: bool = False, device="cuda"):
        self.dims = dims
        self.P = dmoe_padded_rows_max(dims)
        self.map = SparseMap(dims, device)
        u8 = dict(dtype=torch.uint8, device=device)
        self.ws_map = torch.empty(max(dmoe_workspace_bytes(dims, WS_MAP), 16), **u8)
        self.train = train
        P, h, f = self.P, dims.hidden, dims.ffn
        nsc = scale_stride(h)
        bf = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.saved = self.ws_bwd = None
        self.step = {}
        if train:
            total, offs = dmoe_saved_bytes(dims)
            self.saved = torch.empty(total, **u8)
            self.offsets = dict(x_pad=offs[0], a=offs[1], bm=offs[2])
            if dims.flags & SAVE_X_ONLY:  # A and Bm are not saved
                del self.offsets["a"], self.offsets["bm"]
            self.ws_fwd = torch.empty(dmoe_workspace_bytes(dims, WS_FORWARD_TRAIN), **u8)
            self.ws_bwd = torch.empty(max(dmoe_workspace_bytes(dims, WS_BACKWARD), 16), **u8)
            nt = (f + DGLU_TILE_COLS - 1) // DGLU_TILE_COLS
            self.bstep = dict(dy_pad=torch.empty((P, h), **bf), da=torch.empty((P, f), **bf),
                              dbm=torch.empty((P, f), **bf), hw=torch.empty((P, f), **bf),
                              dw_part=torch.empty((P, nt), **f32),
                              dx_pad=torch.empty((P, h), dtype=torch.float16, device=device),
                              dx_scale=torch.empty((P, nsc), **f32))
        else:
            self.ws_fwd = torch.empty(dmoe_workspace_bytes(dims, WS_FORWARD), **u8)
            self.step = dict(x_pad=torch.empty((P, h), **bf), h=torch.empty((P, f), **bf),
                             y_pad=torch.empty((P, h), dtype=torch.float16, device=device),
                             y_scale=torch.empty((P, nsc), **f32),
                             y_acc=torch.empty((dims.T, h), **f32))

    def view(self, name: str) -> torch.Tensor:
        """[P, cols] view of a saved activation (x_pad, a, bm) or, after a training forward,
        of its workspace (h, y_pad, y_scale)."""
        if not self.train:
            return self.step[name]
        P, h, f = self.P, self.dims.hidden, self.dims.ffn
        if name in self.offsets:
            cols = h if name == "x_pad" else f
            off = self.offsets[name]
            return self.saved[off:off + P * cols * 2].view(torch.bfloat16).view(P, cols)
        # forward workspace layout: H [P,f] bf16 | Y_pad [P,h] fp16 | scales [P, scale_stride(h)]
        # fp32, each start aligned to 256 bytes
        up = lambda v: (v + 255) // 256 * 256
        nsc = scale_stride(h)
        o_y = up(P * f * 2)
        o_s = up(o_y + P * h * 2)
        if name == "h":
            return self.ws_fwd[:P * f * 2].view(torch.bfloat16).view(P, f)
        if name == "y_acc" and self.dims.flags & FUSED_COMBINE:  # [T,h] fp32 after H
            T = self.dims.T
            return self.ws_fwd[o_y:o_y + T * h * 4].view(torch.float32).view(T, h)
        if name == "y_pad":
            return self.ws_fwd[o_y:o_y + P * h * 2].view(torch.float16).view(P, h)
        if name == "y_scale":
            return self.ws_fwd[o_s:o_s + P * nsc * 4].view(torch.float32).view(P, nsc)
        raise KeyError(f"{name} is not saved with these flags")
