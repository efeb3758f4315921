"""GB300-native 4-bit groupwise-affine mixture-of-experts layer (sm_103a).

Thin Python binding over the C ABI in include/moe.h, include/moe_mx.h (MXFP4
weights) and include/moe_blk.h (block-scaled 8-bit weights, the RMS norm).  The functions carry the C names and only marshal arguments (torch
tensors -> device pointers, the current CUDA stream); every step of the layer runs
in the CUDA library.  There is no fallback: if the library is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libbitmoe.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_NONFINITE"}

# Every symbol the headers in include/ declare.
EXPORTED = ("moe_status_string", "moe_device_sm_count", "moe_prepack_bytes", "moe_prepack_codes",
            "moe_prepack_codes_bits", "moe_prepack_scales", "moe_dequant_experts",
            "moe_route_max_blocks", "moe_route_workspace_bytes", "moe_route", "moe_route_noalloc",
            "moe_route_noalloc_check_status",
            "moe_router_logits", "moe_route_x", "moe_layer_x", "moe_topk_wide",
            "moe_forward_workspace_bytes",
            "moe_forward", "moe_layer_workspace_bytes", "moe_layer", "moe_check_status", "moe_profile_enable", "moe_profile_kernel_count",
            "moe_profile_kernel_name", "moe_profile_read", "moe_profile_reset", "moe_debug_decode",
            "moe_route_scored", "moe_mx_scale_bytes", "moe_mx_prepack_scales", "moe_mx_quantize", "moe_mx_dequant",
            "moe_mx_matmul", "moe_mx_linear_workspace_bytes", "moe_mx_linear", "moe_mx_forward_workspace_bytes",
            "moe_mx_forward", "moe_mx_layer_workspace_bytes", "moe_mx_layer",
            "moe_blk_quantize", "moe_blk_quantize_weights", "moe_blk_dequant", "moe_blk_dequant_weights",
            "moe_blk_matmul", "moe_blk_linear_workspace_bytes", "moe_blk_linear", "moe_rmsnorm",
            "moe_blk_forward_workspace_bytes", "moe_blk_forward", "moe_blk_layer_workspace_bytes", "moe_blk_layer")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")
        self.status = status


class _QMat(C.Structure):
    _fields_ = [("q", C.c_void_p), ("sb", C.c_void_p)]


class _Experts(C.Structure):
    _fields_ = [("gate", _QMat), ("up", _QMat), ("down", _QMat), ("n_experts", C.c_int), ("bits", C.c_int)]


class _Routing(C.Structure):
    _fields_ = [("ids", C.c_void_p), ("w", C.c_void_p), ("counts", C.c_void_p), ("offsets", C.c_void_p),
                ("perm", C.c_void_p), ("inv_perm", C.c_void_p), ("block_map", C.c_void_p),
                ("num_blocks", C.c_void_p), ("block_rows", C.c_int)]


class _Scoring(C.Structure):
    _fields_ = [("score", C.c_int), ("bias", C.c_void_p), ("n_group", C.c_int), ("topk_group", C.c_int),
                ("group_top", C.c_int), ("renormalize", C.c_int), ("scale", C.c_float)]


class _MxMat(C.Structure):
    _fields_ = [("q", C.c_void_p), ("sp", C.c_void_p)]


class _MxExperts(C.Structure):
    _fields_ = [("gate", _MxMat), ("up", _MxMat), ("down", _MxMat), ("n_experts", C.c_int)]


class _BlkMat(C.Structure):
    _fields_ = [("q", C.c_void_p), ("s", C.c_void_p)]


class _BlkExperts(C.Structure):
    _fields_ = [("gate", _BlkMat), ("up", _BlkMat), ("down", _BlkMat), ("n_experts", C.c_int)]


_lib_handle = None


def lib(path: Optional[str] = None):
    """Loads the CUDA library (raises if it has not been built).  The environment
    variable BITMOE_LIB may name another build of it (for A/B comparisons)."""
    global _lib_handle
    if _lib_handle is None:
        p = path or os.environ.get("BITMOE_LIB") or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library not built: {p} (run __graft_entry__.build())")
        L = C.CDLL(p)
        L.moe_status_string.restype = C.c_char_p
        L.moe_status_string.argtypes = [C.c_int]
        L.moe_device_sm_count.restype = C.c_int
        L.moe_prepack_bytes.restype = C.c_size_t
        L.moe_prepack_bytes.argtypes = [C.c_int, C.c_int, C.c_int]
        L.moe_prepack_codes.restype = C.c_int
        L.moe_prepack_codes.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]
        L.moe_prepack_codes_bits.restype = C.c_int
        L.moe_prepack_codes_bits.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]
        L.moe_prepack_scales.restype = C.c_int
        L.moe_prepack_scales.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]
        L.moe_route_max_blocks.restype = C.c_int
        L.moe_route_max_blocks.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int]
        L.moe_route_workspace_bytes.restype = C.c_size_t
        L.moe_route_workspace_bytes.argtypes = [C.c_int, C.c_int, C.c_int]
        L.moe_route.restype = C.c_int
        L.moe_route.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(_Routing),
                                C.c_void_p, C.c_size_t, C.c_void_p]
        L.moe_router_logits.restype = C.c_int
        L.moe_router_logits.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p]
        L.moe_route_x.restype = C.c_int
        L.moe_route_x.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                  C.POINTER(_Routing), C.c_void_p, C.c_size_t, C.c_void_p]
        L.moe_topk_wide.restype = C.c_int
        L.moe_topk_wide.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p]
        L.moe_dequant_experts.restype = C.c_int
        L.moe_dequant_experts.argtypes = [C.POINTER(_QMat), C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]
        L.moe_route_noalloc.restype = C.c_int
        L.moe_route_noalloc.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(_Routing),
                                        C.c_void_p]
        L.moe_route_noalloc_check_status.restype = C.c_int
        L.moe_route_noalloc_check_status.argtypes = [C.c_void_p]
        L.moe_forward_workspace_bytes.restype = C.c_size_t
        L.moe_forward_workspace_bytes.argtypes = [C.c_int] * 6
        L.moe_forward.restype = C.c_int
        L.moe_forward.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(_Experts),
                                  C.POINTER(_Experts), C.c_int, C.POINTER(_Routing), C.c_void_p, C.c_void_p,
                                  C.c_size_t, C.c_void_p]
        L.moe_layer_workspace_bytes.restype = C.c_size_t
        L.moe_layer_workspace_bytes.argtypes = [C.c_int] * 6
        L.moe_layer.restype = C.c_int
        L.moe_layer.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int,
                                C.POINTER(_Experts), C.POINTER(_Experts), C.c_int, C.POINTER(_Routing), C.c_void_p,
                                C.c_void_p, C.c_size_t, C.c_void_p]
        L.moe_layer_x.restype = C.c_int
        L.moe_layer_x.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                  C.POINTER(_Experts), C.POINTER(_Experts), C.c_int, C.c_void_p, C.POINTER(_Routing),
                                  C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
        L.moe_check_status.restype = C.c_int
        L.moe_check_status.argtypes = [C.c_void_p, C.c_void_p]
        L.moe_profile_enable.restype = C.c_int
        L.moe_profile_enable.argtypes = [C.c_int]
        L.moe_profile_kernel_count.restype = C.c_int
        L.moe_profile_kernel_name.restype = C.c_char_p
        L.moe_profile_kernel_name.argtypes = [C.c_int]
        L.moe_profile_read.restype = C.c_int
        L.moe_profile_read.argtypes = [C.c_int, C.POINTER(C.c_double), C.POINTER(C.c_longlong)]
        L.moe_profile_reset.restype = None
        L.moe_debug_decode.restype = C.c_int
        L.moe_debug_decode.argtypes = [C.c_longlong, C.c_int]
        i, p, sz, mat = C.c_int, C.c_void_p, C.c_size_t, C.POINTER(_MxMat)
        ex = C.POINTER(_MxExperts)
        blk, bex, ll = C.POINTER(_BlkMat), C.POINTER(_BlkExperts), C.c_longlong
        for name, restype, argtypes in (
                ("moe_route_scored", i, [p, C.POINTER(_Scoring), i, i, i, i, C.POINTER(_Routing), p, sz, p]),
                ("moe_mx_scale_bytes", sz, [i, i, i]),
                ("moe_mx_prepack_scales", i, [p, i, i, i, p, p]),
                ("moe_mx_quantize", i, [p, i, i, i, C.c_longlong, mat, p]),
                ("moe_mx_dequant", i, [mat, i, i, i, i, p, p]),
                ("moe_mx_matmul", i, [mat, i, mat, i, i, p, i, p, sz, p]),
                ("moe_mx_linear_workspace_bytes", sz, [i, i, i]),
                ("moe_mx_linear", i, [p, i, i, i, C.c_longlong, mat, i, p, i, p, sz, p]),
                ("moe_mx_forward_workspace_bytes", sz, [i] * 7),
                ("moe_mx_forward", i, [p, i, i, i, i, ex, ex, i, C.POINTER(_Routing), p, p, sz, p]),
                ("moe_mx_layer_workspace_bytes", sz, [i] * 7),
                ("moe_mx_layer", i, [p, C.POINTER(_Scoring), p, i, i, i, i, i, ex, ex, i, C.POINTER(_Routing), p, p,
                                     sz, p]),
                ("moe_blk_quantize", i, [p, i, i, i, ll, blk, p]),
                ("moe_blk_quantize_weights", i, [p, i, i, i, i, blk, p]),
                ("moe_blk_dequant", i, [blk, i, i, i, p, p]),
                ("moe_blk_dequant_weights", i, [blk, i, i, i, i, p, p]),
                ("moe_blk_matmul", i, [blk, i, blk, i, i, p, i, p, sz, p]),
                ("moe_blk_linear_workspace_bytes", sz, [i, i, i]),
                ("moe_blk_linear", i, [p, i, i, i, ll, blk, i, p, i, p, sz, p]),
                ("moe_rmsnorm", i, [p, i, i, i, ll, p, p, i, p, i, C.c_float, p, i, blk, p]),
                ("moe_blk_forward_workspace_bytes", sz, [i] * 7),
                ("moe_blk_forward", i, [p, blk, i, i, i, i, bex, bex, i, C.POINTER(_Routing), p, p, sz, p]),
                ("moe_blk_layer_workspace_bytes", sz, [i] * 7),
                ("moe_blk_layer", i, [p, C.POINTER(_Scoring), p, blk, i, i, i, i, i, bex, bex, i, C.POINTER(_Routing), p,
                                      p, sz, p])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = restype, argtypes
        _lib_handle = L
    return _lib_handle


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


_raw_stream = _raw_device = None  # the current stream's raw handle of a device, and the current device; from the first call


def _find_stream_calls() -> None:
    global _raw_stream, _raw_device
    import torch
    torch.cuda.current_device()  # initialises CUDA, which the calls below take for granted
    # the handle without building a Stream object (~0.2 against ~3 us)
    _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        _find_stream_calls()
    return _raw_stream(_raw_device())


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


# ----------------------------------------------------------------------- data holders

@dataclasses.dataclass
class QMat:
    """One stacked packed matrix on the device: q int32 [E][K/64][N][2 bits] (group-major codes),
    sb int32 [E][K/64][N]."""
    q: "object"
    sb: "object"

    def _c(self) -> _QMat:
        # the C struct is built once and reused while q and sb are the same tensors (a call marshals
        # three matrices per expert set; rebuilding them cost several microseconds per call)
        c = self.__dict__.get("_cc")
        if c is None or c[0] is not self.q or c[1] is not self.sb:
            c = (self.q, self.sb, _QMat(_ptr(self.q), _ptr(self.sb)))
            self.__dict__["_cc"] = c
        return c[2]


@dataclasses.dataclass
class Experts:
    gate: QMat
    up: QMat
    down: QMat

    @property
    def n_experts(self) -> int:
        return int(self.gate.sb.shape[0])

    @property
    def I(self) -> int:
        return int(self.gate.sb.shape[2])

    @property
    def bits(self) -> int:
        """Bits per code: the prepacked rows hold 2 x bits words per group."""
        return int(self.gate.q.shape[3]) // 2

    def _c(self) -> _Experts:
        # rebuilt only when a matrix or one of its tensors was replaced (identity checks only)
        c = self.__dict__.get("_cc")
        g, u, dn = self.gate, self.up, self.down
        if (c is None or c[0] is not g or c[1] is not u or c[2] is not dn or c[3] is not g.q or c[4] is not g.sb
                or c[5] is not u.q or c[6] is not u.sb or c[7] is not dn.q or c[8] is not dn.sb):
            c = (g, u, dn, g.q, g.sb, u.q, u.sb, dn.q, dn.sb,
                 _Experts(g._c(), u._c(), dn._c(), self.n_experts, self.bits), self.I)
            self.__dict__["_cc"] = c
        return c[9]

    def _c_and_I(self):
        """The C struct and the intermediate width, from the same cache."""
        st = self._c()
        return st, self.__dict__["_cc"][10]


_READS, _READS_IDS, _WRITES = range(3)  # what a call does with a Routing's buffers


@dataclasses.dataclass
class Routing:
    """Device buffers written by moe_route, as large as include/moe.h says or larger: a call that needs more than there
    is raises ValueError."""
    ids: "object"
    w: "object"
    counts: "object"
    offsets: "object"
    perm: "object"
    inv_perm: "object"
    block_map: "object"
    num_blocks: "object"
    block_rows: int

    @staticmethod
    def empty(T: int, E: int, k: int, block_rows: int, device="cuda") -> "Routing":
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        A = T * k
        mb = max(1, moe_route_max_blocks(T, E, k, block_rows))
        return Routing(ids=torch.empty((T, k), **i32), w=torch.empty((T, k), dtype=torch.float32, device=device),
                       counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                       perm=torch.empty(max(A, 1), **i32), inv_perm=torch.empty(max(A, 1), **i32),
                       block_map=torch.empty((mb, 3), **i32), num_blocks=torch.zeros(1, **i32),
                       block_rows=block_rows)

    def _cached(self, call=None):
        """The buffers' addresses, the C struct and a reference to it: rebuilt where an address changed.  call: (T, E, k,
        block_rows, use) of a call, for which they have to be large enough."""
        c = self._known
        at = [b.data_ptr() for b in c[4]]
        if c[0] != at:
            every = (self.ids, self.w, self.counts, self.offsets, self.perm, self.inv_perm, self.block_map, self.num_blocks)
            st = _Routing(*(_ptr(b) for b in every), self.block_rows)
            there = [b for b in every if b is not None]
            c = self._known = ([b.data_ptr() for b in there], st, C.byref(st), set(), there)
        c[1].block_rows = self.block_rows
        if call is not None and call not in c[3]:  # (calls found to fit, until a buffer changes)
            self._check(*call)
            if len(c[3]) >= 64:
                c[3].clear()
            c[3].add(call)
        return c

    _known = (None, None, None, None, ())  # addresses, struct, reference, calls, the buffers that there are

    def __setattr__(self, name, value):
        # (a buffer put in another's place may start where that one did and be shorter)
        if name != "block_rows" and name != "_known":
            self.__dict__.pop("_known", None)
        object.__setattr__(self, name, value)

    def _c(self) -> _Routing:
        return self._cached()[1]

    def _check(self, T: int, E: int, k: int, block_rows: int, use: int) -> None:
        """The buffers that a call uses (_WRITES: all; _READS_IDS, _READS: what expert calls may read) are as large as
        include/moe.h says."""
        A = T * k
        tiles = -(-A // block_rows) + E if A > 0 and block_rows > 0 else 0
        need = [("w", A), ("perm", A), ("inv_perm", A), ("block_map", 3 * tiles), ("num_blocks", 1)]
        if use >= _READS_IDS:
            need.append(("ids", A))
        if use == _WRITES:
            need += [("counts", E), ("offsets", E + 1)]
        for name, n in need:
            b = getattr(self, name)
            if b is None:  # the library refuses the call where it needs it
                continue
            if not b.is_cuda or b.element_size() != 4 or not b.is_contiguous():
                raise ValueError(f"routing: {name} ({b.dtype} on {b.device}), expected contiguous 32-bit values on a CUDA device")
            if b.numel() < n:
                raise ValueError(f"routing: {name} has {b.numel()} elements, expected {n} or more for {T} tokens, "
                                 f"{k} of {E} experts each, in tiles of {block_rows} rows")


def workspace(nbytes: int, device="cuda"):
    """A zero-filled, 256-byte aligned device workspace."""
    import torch
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------------- the C functions

def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def moe_device_sm_count() -> int:
    return int(lib().moe_device_sm_count())


def moe_prepack_bytes(E: int, N: int, K: int) -> int:
    return int(lib().moe_prepack_bytes(E, N, K))


def moe_prepack_codes(q, qp, stream=None, bits: int = 4) -> None:
    """q int32 [E][N][K*bits/32] (row-major codes) -> qp int32 [E][K/64][N][2 bits] (group-major)."""
    E, N, W = q.shape
    K = W * 32 // bits
    _check("moe_prepack_codes_bits", lib().moe_prepack_codes_bits(_ptr(q), E, N, K, bits, _ptr(qp), _stream(stream)))


def moe_prepack_scales(scale, bias, sb, stream=None) -> None:
    """scale, bias: int16/uint16-bit [E][N][K/64] device tensors; sb: int32 [E][K/64][N]."""
    E, N, G = scale.shape
    assert bias.shape == scale.shape and tuple(sb.shape) == (E, G, N)
    _check("moe_prepack_scales",
           lib().moe_prepack_scales(_ptr(scale), _ptr(bias), E, N, G * 64, _ptr(sb), _stream(stream)))


def moe_route_max_blocks(T: int, E: int, k: int, block_rows: int) -> int:
    return int(lib().moe_route_max_blocks(T, E, k, block_rows))


def moe_route_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(lib().moe_route_workspace_bytes(T, E, k))


def moe_route(logits, k: int, block_rows: int, out: Routing, ws, stream=None) -> None:
    T, E = logits.shape
    r = out._cached((T, E, k, block_rows, _WRITES))[1]
    _check("moe_route", lib().moe_route(_ptr(logits), T, E, k, block_rows, C.byref(r), _ptr(ws), ws.numel(),
                                        _stream(stream)))
    out.block_rows = r.block_rows


def moe_router_logits(X, W_r, logits, stream=None) -> None:
    """logits [T][E] fp32 = X [T][d] bf16 (int16 storage) times W_r [E][d] bf16, transposed."""
    T, d = X.shape
    E = W_r.shape[0]
    _check("moe_router_logits", lib().moe_router_logits(_ptr(X), T, d, _ptr(W_r), E, _ptr(logits), _stream(stream)))


def moe_route_x(X, W_r, k: int, block_rows: int, out: Routing, ws, logits, stream=None) -> None:
    """moe_router_logits into `logits`, then moe_route on them."""
    T, d = X.shape
    E = W_r.shape[0]
    r = out._cached((T, E, k, block_rows, _WRITES))[1]
    _check("moe_route_x", lib().moe_route_x(_ptr(X), T, d, _ptr(W_r), E, k, block_rows, _ptr(logits), C.byref(r),
                                            _ptr(ws), ws.numel(), _stream(stream)))
    out.block_rows = r.block_rows


def moe_topk_wide(logits, K: int, values, indices, stream=None) -> None:
    """values [T][K] fp32 and indices [T][K] int32: each row's K largest entries of logits [T][V]."""
    T, V = logits.shape
    _check("moe_topk_wide", lib().moe_topk_wide(_ptr(logits), T, V, K, _ptr(values), _ptr(indices), _stream(stream)))


def moe_route_noalloc(logits, k: int, block_rows: int, out: Routing, stream=None) -> None:
    """moe_route without a workspace (for callers that cannot allocate device
    memory): uses the library's built-in scratch array; calls must not overlap
    on the GPU."""
    T, E = logits.shape
    r = out._cached((T, E, k, block_rows, _WRITES))[1]
    _check("moe_route_noalloc", lib().moe_route_noalloc(_ptr(logits), T, E, k, block_rows, C.byref(r),
                                                        _stream(stream)))
    out.block_rows = r.block_rows


def moe_route_noalloc_check_status(stream=None) -> int:
    """Synchronises; the first device-side error recorded by moe_route_noalloc
    calls on the current device since the last check (0 if none), cleared."""
    return int(lib().moe_route_noalloc_check_status(_stream(stream)))


def moe_forward_workspace_bytes(T: int, d: int, I: int, E: int, k: int, I_shared: int) -> int:
    return int(lib().moe_forward_workspace_bytes(T, d, I, E, k, I_shared))


def moe_forward(X, routed: Experts, shared: Optional[Experts], routing: Routing, Y, ws, stream=None) -> None:
    T, d = X.shape
    k = int(routing.ids.shape[1])
    re = routed._c()
    se = shared._c() if shared is not None else None
    I_sh = shared.I if shared is not None else 0
    rr = routing._cached((T, re.n_experts, k, routing.block_rows, _READS_IDS))[1]
    _check("moe_forward", lib().moe_forward(_ptr(X), T, d, routed.I, k, C.byref(re),
                                            C.byref(se) if se is not None else None, I_sh, C.byref(rr), _ptr(Y),
                                            _ptr(ws), ws.numel(), _stream(stream)))


def moe_layer_workspace_bytes(T: int, d: int, I: int, E: int, k: int, I_shared: int) -> int:
    return int(lib().moe_layer_workspace_bytes(T, d, I, E, k, I_shared))


def moe_layer(logits, X, routed: Experts, shared: Optional[Experts], k: int, block_rows: int, out: Routing, Y, ws,
              stream=None) -> None:
    """moe_route + moe_forward in one call (one launch on the decode path)."""
    T, d = X.shape
    re, I = routed._c_and_I()
    se, I_sh = shared._c_and_I() if shared is not None else (None, 0)
    r = out._cached((T, re.n_experts, k, block_rows, _WRITES))[1]
    _check("moe_layer", lib().moe_layer(_ptr(logits), _ptr(X), T, d, I, k, block_rows, C.byref(re),
                                        C.byref(se) if se is not None else None, I_sh, C.byref(r), _ptr(Y),
                                        _ptr(ws), ws.numel(), _stream(stream)))
    out.block_rows = r.block_rows


def moe_layer_x(X, W_r, routed: Experts, shared: Optional[Experts], k: int, block_rows: int, logits, out: Routing,
                Y, ws, stream=None) -> None:
    """moe_router_logits into `logits`, then moe_layer on them: the layer from the hidden state."""
    T, d = X.shape
    re = routed._c()
    se = shared._c() if shared is not None else None
    I_sh = shared.I if shared is not None else 0
    r = out._cached((T, re.n_experts, k, block_rows, _WRITES))[1]
    _check("moe_layer_x", lib().moe_layer_x(_ptr(X), T, d, _ptr(W_r), routed.I, k, block_rows, C.byref(re),
                                            C.byref(se) if se is not None else None, I_sh, _ptr(logits), C.byref(r),
                                            _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)))
    out.block_rows = r.block_rows


def moe_check_status(ws, stream=None) -> int:
    return int(lib().moe_check_status(_ptr(ws), _stream(stream)))


def moe_profile_enable(on: bool) -> bool:
    return bool(lib().moe_profile_enable(1 if on else 0))


def moe_profile_reset() -> None:
    lib().moe_profile_reset()


def moe_debug_decode(wait_limit_cycles: int = 0, drop_cta: int = -1) -> None:
    """Test hook of the decode kernel: the limit of the wait at its barrier over
    the grid (cycles, 0 = default) and a CTA whose arrival there is skipped."""
    _check("moe_debug_decode", lib().moe_debug_decode(int(wait_limit_cycles), int(drop_cta)))


def moe_profile_read() -> dict:
    """{kernel name: (total device ms, launches)} for every kernel kind timed since the last reset."""
    L = lib()
    out = {}
    for i in range(L.moe_profile_kernel_count()):
        ms = C.c_double()
        n = C.c_longlong()
        _check("moe_profile_read", L.moe_profile_read(i, C.byref(ms), C.byref(n)))
        out[L.moe_profile_kernel_name(i).decode()] = (ms.value, n.value)
    return out


# ----------------------------------------------------------------------- scored routing, MXFP4

SCORES = {"softmax": 0, "sigmoid": 1}


@dataclasses.dataclass
class Scoring:
    """How moe_route_scored scores a token's logits (see include/moe.h): softmax or sigmoid scores, a bias for the
    selection (fp32 [E] on the device, or None), groups, weights renormalised over the selection and scaled."""
    score: str = "softmax"
    bias: "object" = None
    n_group: int = 1
    topk_group: int = 1
    group_top: int = 2
    renormalize: bool = True
    scale: float = 1.0

    def _ref(self, E: int):
        """A reference to the C struct, rebuilt only when a field or the bias's address changed."""
        c = self.__dict__.get("_cc")
        key = (self.score, self.n_group, self.topk_group, self.group_top, self.renormalize, self.scale, E, _ptr(self.bias))
        if c is None or c[0] is not self.bias or c[1] != key:
            if self.score not in SCORES:
                raise ValueError(f"score {self.score!r}: one of {sorted(SCORES)}")
            if self.bias is not None:
                _tensor("bias", self.bias, (_FP32,), (E,))
            top = 1 if self.n_group == 1 else self.group_top
            c = (self.bias, key, C.byref(_Scoring(SCORES[self.score], _ptr(self.bias), self.n_group, self.topk_group,
                                                  top, 1 if self.renormalize else 0, self.scale)))
            self.__dict__["_cc"] = c
        return c[2]


_BF16, _FP16, _FP32, _U8, _E4M3 = 0, 1, 2, 3, 4  # the first three as moe_dtype
_DTYPE_NAMES = {"bfloat16": _BF16, "int16": _BF16, "float16": _FP16, "float32": _FP32, "uint8": _U8, "float8_e4m3fn": _E4M3}
_dtype_codes = {}  # torch.dtype -> code, filled as types are met


def _code(t) -> int:
    """The type code of a tensor (int16 stands for bf16 bit patterns), -1 for another type."""
    d = t.dtype
    c = _dtype_codes.get(d)
    if c is None:
        c = _dtype_codes[d] = _DTYPE_NAMES.get(str(d)[6:], -1)  # "torch.float32" -> "float32"
    return c


def _tensor(name: str, t, codes, shape=None) -> int:
    """The type code of t, a contiguous CUDA tensor of one of the types and, where given, of the shape."""
    c = _dtype_codes.get(t.dtype)
    if c is None:
        c = _code(t)
    if c not in codes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(n for n, v in _DTYPE_NAMES.items() if v in codes)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    return c


_FLOATS = (_BF16, _FP16, _FP32)
_ONLY_BF16, _ONLY_FP32 = (_BF16,), (_FP32,)


def _rows(name: str, t):
    """(rows, columns, elements between rows, type code) of a 2-D CUDA tensor with contiguous rows."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name}: expected a 2-D CUDA tensor, got {tuple(shape)} on {t.device}")
    rows, cols = shape
    code = _dtype_codes.get(t.dtype)
    if code is None:
        code = _code(t)
    if code not in _FLOATS:
        raise ValueError(f"{name}: {t.dtype}, expected bfloat16, int16 (bf16 bits), float16 or float32")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: elements of a row are {step} apart, expected 1")
    return rows, cols, (ld if rows > 1 else cols), code


def moe_mx_scale_bytes(E: int, N: int, K: int) -> int:
    return int(lib().moe_mx_scale_bytes(E, N, K))


@dataclasses.dataclass
class MxMat:
    """A stack of MXFP4 matrices on the device: q uint8 [E][N][K/2] (two codes a byte, the lower column in the low
    nibble), sp uint8 [E][ceil(N/128)][ceil(K/128)][512] (packed scales, see include/moe_mx.h)."""
    q: "object"
    sp: "object"

    @staticmethod
    def empty(E: int, N: int, K: int, device="cuda") -> "MxMat":
        """Room for E matrices, e.g. as the result of moe_mx_quantize (E = 1)."""
        import torch
        n = moe_mx_scale_bytes(E, N, K)
        if n == 0:
            raise ValueError(f"no MXFP4 matrices of E={E}, N={N}, K={K}: K is a positive multiple of 32")
        return MxMat(torch.empty((E, N, K // 2), dtype=torch.uint8, device=device),
                     torch.empty((E, -(-N // 128), -(-K // 128), 512), dtype=torch.uint8, device=device))

    @property
    def shape(self):
        """(E, N, K)"""
        E, N, half = self.q.shape
        return int(E), int(N), 2 * int(half)

    _known = (None, None, 0, 0, None, 0, None)  # q, sp, their addresses, q's shape, sp's size, what _ref_and_shape gives

    def _ref_and_shape(self):
        """A reference to the C struct, (E, N, K), and the struct: rebuilt where a tensor, its memory or layout changed."""
        q, sp = self.q, self.sp
        kq, ks, aq, asp, qshape, size, known = self._known
        if (q is not kq or sp is not ks or q.data_ptr() != aq or sp.data_ptr() != asp or q.shape != qshape
                or sp.numel() != size or not q.is_contiguous()):
            _tensor("q", q, (_U8,))
            if q.dim() != 3:
                raise ValueError(f"q: shape {tuple(q.shape)}, expected [E][N][K/2]")
            E, N, K = self.shape
            _tensor("sp", sp, (_U8,), (E, -(-N // 128), -(-K // 128), 512))
            st = _MxMat(_ptr(q), _ptr(sp))
            known = (C.byref(st), (E, N, K), st)
            self._known = (q, sp, st.q, st.sp, q.shape, sp.numel(), known)
        return known

    def _c(self) -> _MxMat:
        return self._ref_and_shape()[2]


@dataclasses.dataclass
class MxExperts:
    """One expert set: gate and up [E][I][d], down [E][d][I]."""
    gate: MxMat
    up: MxMat
    down: MxMat

    def _ref_and_sizes(self):
        """A reference to the C struct, and (E, I, d)."""
        # rebuilt where a matrix's was: that is the same object until then
        g, u, dn = self.gate._ref_and_shape(), self.up._ref_and_shape(), self.down._ref_and_shape()
        kg, ku, kd, known = self._known
        if g is not kg or u is not ku or dn is not kd:
            E, I, d = g[1]
            if u[1] != (E, I, d) or dn[1] != (E, d, I):
                raise ValueError(f"gate {g[1]}, up {u[1]}, down {dn[1]}: expected (E, I, d) twice and (E, d, I)")
            known = (C.byref(_MxExperts(g[2], u[2], dn[2], E)), (E, I, d))
            self._known = (g, u, dn, known)
        return known

    _known = (None, None, None, None)


def moe_route_scored(logits, scoring: Scoring, k: int, block_rows: int, out: Routing, ws, stream=None) -> None:
    """moe_route with softmax or sigmoid scores, a selection bias and groups (fp32 logits [T][E])."""
    _tensor("logits", logits, _ONLY_FP32)
    T, E = logits.shape
    r = out._cached((T, E, k, block_rows, _WRITES))[2]
    status = lib().moe_route_scored(logits.data_ptr(), scoring._ref(E), T, E, k, block_rows, r, ws.data_ptr(),
                                    ws.numel(), _stream(stream))
    if status:
        _check("moe_route_scored", status)
    out.block_rows = block_rows


def moe_mx_prepack_scales(scale, sp, stream=None) -> None:
    """scale uint8 [E][N][K/32] (E8M0, row-major) -> sp [E][ceil(N/128)][ceil(K/128)][512]."""
    _tensor("scale", scale, (_U8,))
    E, N, G = scale.shape
    _tensor("sp", sp, (_U8,), (E, -(-N // 128), -(-G // 4), 512))
    status = lib().moe_mx_prepack_scales(_ptr(scale), E, N, 32 * G, _ptr(sp), _stream(stream))
    if status:
        _check("moe_mx_prepack_scales", status)


def moe_mx_quantize(X, out: MxMat, stream=None) -> None:
    """X [rows][K] (bf16, fp16 or fp32; rows may be strided) -> out, an MxMat of (1, rows, K).

    A product that takes `out` as its weights may be the next call on the stream."""
    rows, K, ld, code = _rows("X", X)
    m, shape, _ = out._ref_and_shape()
    if shape != (1, rows, K):
        raise ValueError(f"out: {shape}, expected (1, {rows}, {K})")
    status = lib().moe_mx_quantize(X.data_ptr(), code, rows, K, ld, m, _stream(stream))
    if status:
        _check("moe_mx_quantize", status)


def moe_mx_dequant(m: MxMat, W, stream=None) -> None:
    """W (bf16 or fp32, E*N*K elements) = the values of m."""
    ref, (E, N, K), _ = m._ref_and_shape()
    code = _tensor("W", W, _FLOATS)
    if W.numel() != E * N * K:
        raise ValueError(f"W: {W.numel()} elements, expected {E * N * K}")
    status = lib().moe_mx_dequant(ref, E, N, K, code, W.data_ptr(), _stream(stream))
    if status:
        _check("moe_mx_dequant", status)


def _one(name: str, W: MxMat):
    ref, (E, N, K), _ = W._ref_and_shape()
    if E != 1:
        raise ValueError(f"{name}: {E} matrices, expected one")
    return ref, N, K


def moe_mx_matmul(A: MxMat, W: MxMat, Y, ws, stream=None) -> None:
    """Y [M][N] (bf16 or fp32) = A (1, M, K) times W (1, N, K), transposed."""
    a, M, K = _one("A", A)
    w, N, Kw = _one("W", W)
    if K != Kw:
        raise ValueError(f"A has {K} columns, W {Kw}")
    y = _tensor("Y", Y, _FLOATS, (M, N))
    status = lib().moe_mx_matmul(a, M, w, N, K, Y.data_ptr(), y, ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        _check("moe_mx_matmul", status)


def moe_mx_linear_workspace_bytes(T: int, N: int, K: int) -> int:
    return int(lib().moe_mx_linear_workspace_bytes(T, N, K))


def moe_mx_linear(X, W: MxMat, Y, ws, stream=None) -> None:
    """Y [T][N] = MXFP4(X [T][K]) times W (1, N, K), transposed: a linear layer with MXFP4 weights."""
    T, K, ld, code = _rows("X", X)
    w, N, Kw = _one("W", W)
    if K != Kw:
        raise ValueError(f"X has {K} columns, W {Kw}")
    y = _tensor("Y", Y, _FLOATS, (T, N))
    status = lib().moe_mx_linear(X.data_ptr(), code, T, K, ld, w, N, Y.data_ptr(), y, ws.data_ptr(), ws.numel(),
                                 _stream(stream))
    if status:
        _check("moe_mx_linear", status)


def moe_mx_forward_workspace_bytes(T: int, d: int, I: int, E: int, k: int, I_shared: int, block_rows: int) -> int:
    return int(lib().moe_mx_forward_workspace_bytes(T, d, I, E, k, I_shared, block_rows))


def _mx_sets(X, routed: MxExperts, shared: Optional[MxExperts], Y):
    """References to the C structs and the sizes of an expert call, shapes checked."""
    _tensor("X", X, _ONLY_BF16)
    T, d = shape = X.shape
    re, (E, I, dr) = routed._ref_and_sizes()
    se, I_sh = None, 0
    if shared is not None:
        se, (Es, I_sh, ds) = shared._ref_and_sizes()
        if Es != 1 or ds != d:
            raise ValueError(f"shared: ({Es}, {I_sh}, {ds}), expected one expert of width {d}")
    if dr != d:
        raise ValueError(f"X is {d} wide, the experts {dr}")
    _tensor("Y", Y, _ONLY_BF16, shape)
    return T, d, E, I, I_sh, re, se


def moe_mx_forward(X, routed: MxExperts, shared: Optional[MxExperts], routing: Routing, Y, ws, stream=None) -> None:
    """The expert layer on MXFP4 weights, for a routing of moe_route or moe_route_scored."""
    T, d, E, I, I_sh, re, se = _mx_sets(X, routed, shared, Y)
    k = routing.ids.shape[1]
    rr = routing._cached((T, E, k, routing.block_rows, _READS))[2]
    status = lib().moe_mx_forward(X.data_ptr(), T, d, I, k, re, se, I_sh, rr,
                                  Y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        _check("moe_mx_forward", status)


def moe_mx_layer_workspace_bytes(T: int, d: int, I: int, E: int, k: int, I_shared: int, block_rows: int) -> int:
    return int(lib().moe_mx_layer_workspace_bytes(T, d, I, E, k, I_shared, block_rows))


def moe_mx_layer(logits, scoring: Scoring, X, routed: MxExperts, shared: Optional[MxExperts], k: int, block_rows: int,
                 out: Routing, Y, ws, stream=None) -> None:
    """moe_route_scored + moe_mx_forward in one call."""
    T, d, E, I, I_sh, re, se = _mx_sets(X, routed, shared, Y)
    _tensor("logits", logits, _ONLY_FP32, (T, E))
    r = out._cached((T, E, k, block_rows, _WRITES))[2]
    status = lib().moe_mx_layer(logits.data_ptr(), scoring._ref(E), X.data_ptr(), T, d, I, k, block_rows, re, se, I_sh,
                                r, Y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        _check("moe_mx_layer", status)
    out.block_rows = block_rows


# ----------------------------------------------------------------------- block-scaled 8-bit floating point, RMS norm

_CODES = (_U8, _E4M3)


@dataclasses.dataclass
class _BlkCodes:
    """Codes q (uint8 or float8_e4m3fn) and scales s (fp32) on the device, see include/moe_blk.h."""
    q: "object"
    s: "object"

    _known = (None, None, 0, 0, None, 0, 0, None, None)  # q, s, what they were like, what _ref_and_shape gives

    def _ref_and_shape(self):
        """A reference to the C struct, the shape, and the struct: rebuilt where a tensor, its memory or layout changed."""
        q, s = self.q, self.s
        kq, ks, aq, at, strides, size, sn, stype, known = self._known
        # (the strides of a contiguous q say all but its first size; a stack's is that of s too)
        if (q is not kq or s is not ks or q.data_ptr() != aq or s.data_ptr() != at or q.stride() != strides
                or s.numel() != sn or s.dtype is not stype or self._rows and q.numel() != size):
            _tensor("q", q, _CODES)
            shape, scales = self._shapes()
            _tensor("s", s, _ONLY_FP32, scales)
            aq, at = q.data_ptr(), s.data_ptr()
            st = _BlkMat(aq, at)
            known = (C.byref(st), shape, st)
            self._known = (q, s, aq, at, q.stride(), q.numel(), s.numel(), s.dtype, known)
        return known


class BlkMat(_BlkCodes):
    """A stack of weight matrices: q [E][N][K], s [E][ceil(N/128)][ceil(K/128)], as checkpoints hold them."""
    _rows = False

    @staticmethod
    def empty(E: int, N: int, K: int, device="cuda") -> "BlkMat":
        """Room for E matrices, e.g. as the result of moe_blk_quantize_weights."""
        import torch
        return BlkMat(torch.empty((E, N, K), dtype=torch.uint8, device=device),
                      torch.empty((E, -(-N // 128), -(-K // 128)), dtype=torch.float32, device=device))

    def _shapes(self):
        if self.q.dim() != 3:
            raise ValueError(f"q: shape {tuple(self.q.shape)}, expected [E][N][K]")
        E, N, K = self.q.shape
        return (E, N, K), (E, -(-N // 128), -(-K // 128))


class BlkAct(_BlkCodes):
    """Activations: q [rows][K], s [ceil(K/128)][rows up to a multiple of 4]."""
    _rows = True

    @staticmethod
    def empty(rows: int, K: int, device="cuda") -> "BlkAct":
        """Room for the result of moe_blk_quantize or moe_rmsnorm."""
        import torch
        return BlkAct(torch.empty((rows, K), dtype=torch.uint8, device=device),
                      torch.empty((-(-K // 128), (rows + 3) // 4 * 4), dtype=torch.float32, device=device))

    def _shapes(self):
        if self.q.dim() != 2:
            raise ValueError(f"q: shape {tuple(self.q.shape)}, expected [rows][K]")
        rows, K = self.q.shape
        return (rows, K), (-(-K // 128), (rows + 3) // 4 * 4)


@dataclasses.dataclass
class BlkExperts:
    """One expert set: gate and up [E][I][d], down [E][d][I]."""
    gate: BlkMat
    up: BlkMat
    down: BlkMat

    def _ref_and_sizes(self):
        """A reference to the C struct, and (E, I, d)."""
        # rebuilt where a matrix's was: that is the same object until then
        g, u, dn = self.gate._ref_and_shape(), self.up._ref_and_shape(), self.down._ref_and_shape()
        kg, ku, kd, known = self._known
        if g is not kg or u is not ku or dn is not kd:
            E, I, d = g[1]
            if u[1] != (E, I, d) or dn[1] != (E, d, I):
                raise ValueError(f"gate {g[1]}, up {u[1]}, down {dn[1]}: expected (E, I, d) twice and (E, d, I)")
            known = (C.byref(_BlkExperts(g[2], u[2], dn[2], E)), (E, I, d))
            self._known = (g, u, dn, known)
        return known

    _known = (None, None, None, None)


def moe_blk_quantize(X, out: BlkAct, stream=None) -> None:
    """X [rows][K] (bf16, fp16 or fp32; rows may be strided) -> out: a scale per row and 128 columns."""
    rows, K, ld, code = _rows("X", X)
    m, shape, _ = out._ref_and_shape()
    if type(out) is not BlkAct or shape != (rows, K):
        raise ValueError(f"out: {type(out).__name__} of {shape}, expected BlkAct of ({rows}, {K})")
    status = lib().moe_blk_quantize(X.data_ptr(), code, rows, K, ld, m, _stream(stream))
    if status:
        _check("moe_blk_quantize", status)


def moe_blk_quantize_weights(W, out: BlkMat, stream=None) -> None:
    """W [E][N][K] (bf16, fp16 or fp32) -> out: a scale per block of 128 x 128.

    A product that takes `out` as its weights may be the next call on the stream."""
    code = _tensor("W", W, _FLOATS)
    m, shape, _ = out._ref_and_shape()
    if type(out) is not BlkMat or W.shape != shape:
        raise ValueError(f"out: {type(out).__name__} of {shape}, expected BlkMat of {tuple(W.shape)}")
    status = lib().moe_blk_quantize_weights(W.data_ptr(), code, *shape, m, _stream(stream))
    if status:
        _check("moe_blk_quantize_weights", status)


def moe_blk_dequant(m, X, stream=None) -> None:
    """X (bf16, fp16 or fp32, m's shape) = the values of m, a BlkAct or a BlkMat."""
    ref, shape, _ = m._ref_and_shape()
    code = _tensor("X", X, _FLOATS, shape)
    fn = lib().moe_blk_dequant if type(m) is BlkAct else lib().moe_blk_dequant_weights
    status = fn(ref, *shape, code, X.data_ptr(), _stream(stream))
    if status:
        _check("moe_blk_dequant", status)


def _blk_one(W: BlkMat, K: int):
    ref, shape, _ = W._ref_and_shape()
    if type(W) is not BlkMat or shape[0] != 1:
        raise ValueError(f"W: {type(W).__name__} of {shape}, expected a BlkMat of one matrix")
    if shape[2] != K:
        raise ValueError(f"the activations have {K} columns, W {shape[2]}")
    return ref, shape[1]


def moe_blk_matmul(A: BlkAct, W: BlkMat, Y, ws, stream=None) -> None:
    """Y [M][N] (bf16, fp16 or fp32) = A (M, K) times W (1, N, K), transposed."""
    a, shape, _ = A._ref_and_shape()
    if type(A) is not BlkAct:
        raise ValueError(f"A: {type(A).__name__}, expected BlkAct")
    M, K = shape
    w, N = _blk_one(W, K)
    y = _tensor("Y", Y, _FLOATS, (M, N))
    status = lib().moe_blk_matmul(a, M, w, N, K, Y.data_ptr(), y, ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        _check("moe_blk_matmul", status)


def moe_blk_linear_workspace_bytes(T: int, N: int, K: int) -> int:
    return int(lib().moe_blk_linear_workspace_bytes(T, N, K))


def moe_blk_linear(X, W: BlkMat, Y, ws, stream=None) -> None:
    """Y [T][N] = quantised X [T][K] times W (1, N, K), transposed: a linear layer with block-scaled 8-bit weights."""
    T, K, ld, code = _rows("X", X)
    w, N = _blk_one(W, K)
    y = _tensor("Y", Y, _FLOATS, (T, N))
    status = lib().moe_blk_linear(X.data_ptr(), code, T, K, ld, w, N, Y.data_ptr(), y, ws.data_ptr(), ws.numel(),
                                  _stream(stream))
    if status:
        _check("moe_blk_linear", status)


def moe_rmsnorm(X, gamma, eps: float, residual=None, stream_out=None, Y=None, out: Optional[BlkAct] = None,
                stream=None) -> None:
    """r = X + residual (written to stream_out, by default the residual itself), y = r / sqrt(mean(r^2) + eps) * gamma.

    X [T][d] (bf16, fp16 or fp32; rows may be strided); residual [T][d] of X's type or fp32, or None; gamma [d], bf16 or
    fp32.  y goes to Y [T][d] (bf16, fp16 or fp32), quantised to out, or to both."""
    T, d, ld, code = _rows("X", X)
    shape = X.shape
    rp = op = yp = 0
    rt = yt = code
    if residual is not None:
        rt = _tensor("residual", residual, _FLOATS, shape)
        rp = op = residual.data_ptr()
        if stream_out is not None:
            if _tensor("stream_out", stream_out, _FLOATS, shape) != rt:
                raise ValueError(f"stream_out: {stream_out.dtype}, the residual {residual.dtype}")
            op = stream_out.data_ptr()
    elif stream_out is not None:
        raise ValueError("stream_out without a residual")
    gt = _tensor("gamma", gamma, _GAMMA, (d,))
    if Y is not None:
        yt = _tensor("Y", Y, _FLOATS, shape)
        yp = Y.data_ptr()
    q = None
    if out is not None:
        q, qshape, _ = out._ref_and_shape()
        if type(out) is not BlkAct or qshape != shape:
            raise ValueError(f"out: {type(out).__name__} of {qshape}, expected BlkAct of {tuple(shape)}")
    status = lib().moe_rmsnorm(X.data_ptr(), code, T, d, ld, rp, op, rt, gamma.data_ptr(), gt, eps, yp, yt, q,
                               _stream(stream))
    if status:
        _check("moe_rmsnorm", status)


_GAMMA = (_BF16, _FP32)


def moe_blk_forward_workspace_bytes(T: int, d: int, I: int, E: int, k: int, I_shared: int, block_rows: int) -> int:
    return int(lib().moe_blk_forward_workspace_bytes(T, d, I, E, k, I_shared, block_rows))


def _blk_sets(X, routed: BlkExperts, shared: Optional[BlkExperts], Y):
    """References to the C structs and the sizes of an expert call, shapes checked."""
    if type(X) is BlkAct:
        xq, shape, _ = X._ref_and_shape()
        xp = 0
    else:
        _tensor("X", X, _ONLY_BF16)
        xq, shape, xp = None, X.shape, X.data_ptr()
    T, d = shape
    re, (E, I, dr) = routed._ref_and_sizes()
    se, I_sh = None, 0
    if shared is not None:
        se, (Es, I_sh, ds) = shared._ref_and_sizes()
        if Es != 1 or ds != d:
            raise ValueError(f"shared: ({Es}, {I_sh}, {ds}), expected one expert of width {d}")
    if dr != d:
        raise ValueError(f"X is {d} wide, the experts {dr}")
    _tensor("Y", Y, _ONLY_BF16, shape)
    return T, d, E, I, I_sh, re, se, xp, xq


def moe_blk_forward(X, routed: BlkExperts, shared: Optional[BlkExperts], routing: Routing, Y, ws, stream=None) -> None:
    """The expert layer on block-scaled 8-bit weights; X: bf16 [T][d], or a BlkAct taken as it is."""
    T, d, E, I, I_sh, re, se, xp, xq = _blk_sets(X, routed, shared, Y)
    k = routing.ids.shape[1]
    rr = routing._cached((T, E, k, routing.block_rows, _READS))[2]
    status = lib().moe_blk_forward(xp, xq, T, d, I, k, re, se, I_sh, rr, Y.data_ptr(),
                                   ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        _check("moe_blk_forward", status)


def moe_blk_layer_workspace_bytes(T: int, d: int, I: int, E: int, k: int, I_shared: int, block_rows: int) -> int:
    return int(lib().moe_blk_layer_workspace_bytes(T, d, I, E, k, I_shared, block_rows))


def moe_blk_layer(logits, scoring: Scoring, X, routed: BlkExperts, shared: Optional[BlkExperts], k: int, block_rows: int,
                  out: Routing, Y, ws, stream=None) -> None:
    """moe_route_scored + moe_blk_forward in one call."""
    T, d, E, I, I_sh, re, se, xp, xq = _blk_sets(X, routed, shared, Y)
    _tensor("logits", logits, _ONLY_FP32, (T, E))
    r = out._cached((T, E, k, block_rows, _WRITES))[2]
    status = lib().moe_blk_layer(logits.data_ptr(), scoring._ref(E), xp, xq, T, d, I, k, block_rows, re, se, I_sh, r,
                                 Y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    if status:
        _check("moe_blk_layer", status)
    out.block_rows = block_rows


# ----------------------------------------------------------------------- weight preparation

def moe_dequant_experts(m: QMat, bits: int, W, stream=None) -> None:
    """W fp16 bits [E][N][K] (int16 tensor) = q * scale + bias of the prepacked matrix m."""
    E, G, N = m.sb.shape
    st = m._c()
    _check("moe_dequant_experts", lib().moe_dequant_experts(C.byref(st), int(E), int(N), int(G) * 64, int(bits),
                                                            _ptr(W), _stream(stream)))


def prepare_experts(ex: dict, device="cuda", stream=None) -> Experts:
    """Device copy of one expert set in the kernels' format.

    ex maps "gate", "up", "down" to (q, scale, bias): q uint32/int32 [E][N][K*bits/32]
    (4-, 3- or 2-bit codes, the width following from the shapes), scale and bias
    uint16/int16 bf16 bits [E][N][K/64], as NumPy arrays or torch tensors.  Codes and group parameters are reordered once with
    moe_prepack_codes and moe_prepack_scales (a one-time layout change, like
    loading a checkpoint).
    """
    import numpy as np
    import torch

    def dev(a, np_view, torch_dtype):
        if isinstance(a, np.ndarray):
            return torch.from_numpy(np.ascontiguousarray(a).view(np_view)).to(device)
        return a.to(device=device).view(torch_dtype).contiguous()

    mats = {}
    for name in ("gate", "up", "down"):
        q, s, b = ex[name]
        qd = dev(q, np.int32, torch.int32)
        sd = dev(s, np.int16, torch.int16)
        bd = dev(b, np.int16, torch.int16)
        E, N, G = sd.shape
        bits = 32 * int(qd.shape[2]) // (64 * G)
        if bits not in (2, 3, 4) or bits * 64 * G != 32 * int(qd.shape[2]):
            raise ValueError(f"{name}: codes [E][N][{qd.shape[2]}] do not match {G} groups of 4-, 3- or 2-bit codes")
        sb = torch.empty((E, G, N), dtype=torch.int32, device=device)
        moe_prepack_scales(sd, bd, sb, stream)
        qp = torch.empty((E, G, N, 2 * bits), dtype=torch.int32, device=device)
        moe_prepack_codes(qd, qp, stream, bits)
        del qd
        mats[name] = QMat(qp, sb)
    return Experts(**mats)


def prepare_mx_experts(ex: dict, device="cuda", stream=None) -> MxExperts:
    """Device copy of one MXFP4 expert set.

    ex maps "gate", "up", "down" to (q, scale): q uint8 [E][N][K/2], scale uint8 E8M0 [E][N][K/32], as NumPy arrays or
    torch tensors.  The scales are packed once with moe_mx_prepack_scales; the codes are used as they are.
    """
    import numpy as np
    import torch

    def dev(a):
        return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).to(device).contiguous()

    mats = {}
    for name in ("gate", "up", "down"):
        q, s = (dev(a) for a in ex[name])
        E, N, G = s.shape
        if tuple(q.shape) != (E, N, 16 * G):
            raise ValueError(f"{name}: codes {tuple(q.shape)} do not match scales {tuple(s.shape)}")
        sp = torch.empty((E, -(-N // 128), -(-G // 4), 512), dtype=torch.uint8, device=device)
        moe_mx_prepack_scales(s, sp, stream)
        mats[name] = MxMat(q, sp)
    return MxExperts(**mats)
