"""ctypes binding of liblora_sgmv.so (argument marshalling only).

Every computation runs in the HIP library; this module only turns torch
tensors and numpy arrays into the pointers and sizes of the C ABI declared
in include/lora_sgmv.h, and raises LoraError on a non-zero status. There is
no fallback path: if the library is not built, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblora_sgmv.so")

LORA_OK = 0
LORA_INVALID_ARGUMENT = 1
LORA_UNSUPPORTED = 2
LORA_WORKSPACE_TOO_SMALL = 3
LORA_DEVICE_ERROR = 4

OP_SHRINK, OP_EXPAND, OP_FUSED, OP_BACKWARD = 0, 1, 2, 3
GRAD_ACCUMULATE = 1


class LoraError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[{status}] {msg}")
        self.status = status


class CAdapters(ctypes.Structure):
    _fields_ = [("num_adapters", ctypes.c_int32), ("h_in", ctypes.c_int32),
                ("h_out", ctypes.c_int32), ("A_ptrs", ctypes.c_void_p),
                ("B_ptrs", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("A_ptrs_host", ctypes.c_void_p),
                ("B_ptrs_host", ctypes.c_void_p)]


class CSegments(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_segments", ctypes.c_int32),
                ("seg_starts", ctypes.c_void_p), ("seg_adapter", ctypes.c_void_p),
                ("token_rows", ctypes.c_void_p), ("token_rows_host", ctypes.c_void_p)]


class CGraphAdapters(ctypes.Structure):
    _fields_ = [("num_adapters", ctypes.c_int32), ("h_in", ctypes.c_int32), ("h_out", ctypes.c_int32),
                ("max_rank", ctypes.c_int32), ("A_ptrs", ctypes.c_void_p), ("B_ptrs", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class CQ8(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("ld", ctypes.c_int64), ("exps", ctypes.c_void_p),
                ("ld_exps", ctypes.c_int64), ("rows", ctypes.c_int32), ("width", ctypes.c_int32),
                ("block_rows", ctypes.c_int32)]


EXPORTS = ["lora_segments_from_ids", "lora_workspace_size", "lora_sgmv_shrink", "lora_sgmv_expand",
           "lora_sgmv_fused", "lora_packed_backward", "lora_workspace_size_multi",
           "lora_sgmv_fused_multi", "lora_sgmv_fused_noalloc", "lora_workspace_size_graph",
           "lora_sgmv_fused_graph", "lora_q8_quantize", "lora_q8_dequantize", "lora_q8_matmul",
           "lora_packed_backward_q8", "lora_swiglu", "lora_swiglu_backward", "lora_status_string", "lora_last_error", "lora_version"]
NOALLOC_SCRATCH_BYTES = 16 << 20  # LORA_NOALLOC_SCRATCH_BYTES

_lib = None
_torch = None  # set by load(): the hot calls look it up once per call, not per import statement


def load(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m lora_adapter_batching_amd.build`")
    # torch (which provides the device memory and streams) brings its own HIP
    # runtime; loading it first makes the library bind to that same runtime,
    # so that one HIP runtime serves the process
    import torch
    global _torch
    _torch = torch
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    lib.lora_segments_from_ids.argtypes = [P, ctypes.c_int32, ctypes.c_int32, P, P, P]
    lib.lora_workspace_size.argtypes = [ctypes.c_int, ctypes.POINTER(CAdapters),
                                        ctypes.POINTER(CSegments), ctypes.POINTER(ctypes.c_size_t)]
    lib.lora_sgmv_shrink.argtypes = [P, I64, ctypes.POINTER(CAdapters), ctypes.POINTER(CSegments),
                                     P, I64, P, ctypes.c_size_t, P]
    lib.lora_sgmv_expand.argtypes = [P, I64, ctypes.POINTER(CAdapters), ctypes.POINTER(CSegments),
                                     P, I64, P, ctypes.c_size_t, P]
    lib.lora_sgmv_fused.argtypes = [P, I64, ctypes.POINTER(CAdapters), ctypes.POINTER(CSegments),
                                    P, I64, P, I64, P, ctypes.c_size_t, P]
    lib.lora_packed_backward.argtypes = [P, I64, P, I64, P, I64, ctypes.POINTER(CAdapters),
                                         ctypes.POINTER(CSegments), P, I64, P, P, ctypes.c_uint32,
                                         P, ctypes.c_size_t, P]
    lib.lora_workspace_size_multi.argtypes = [ctypes.c_int32, P, ctypes.POINTER(CSegments),
                                              ctypes.POINTER(ctypes.c_size_t)]
    lib.lora_sgmv_fused_multi.argtypes = [P, I64, ctypes.c_int32, P, ctypes.POINTER(CSegments), P, P,
                                          P, ctypes.c_size_t, P]
    lib.lora_sgmv_fused_noalloc.argtypes = [P, I64, ctypes.POINTER(CAdapters), ctypes.POINTER(CSegments),
                                            P, I64, P, I64, P]
    lib.lora_workspace_size_graph.argtypes = [ctypes.POINTER(CGraphAdapters), ctypes.c_int32,
                                              ctypes.POINTER(ctypes.c_size_t)]
    lib.lora_sgmv_fused_graph.argtypes = [P, I64, ctypes.POINTER(CGraphAdapters), P, ctypes.c_int32, P, I64,
                                          P, ctypes.c_size_t, P]
    Q = P  # address of a CQ8
    lib.lora_q8_quantize.argtypes = [P, I64, Q, Q, P]
    lib.lora_q8_dequantize.argtypes = [Q, P, I64, P]
    lib.lora_q8_matmul.argtypes = [Q, Q, P, I64, ctypes.c_uint32, P]
    lib.lora_packed_backward_q8.argtypes = [Q, P, I64, P, I64, ctypes.POINTER(CAdapters), ctypes.POINTER(CSegments),
                                            P, I64, P, P, ctypes.c_uint32, P, ctypes.c_size_t, P]
    lib.lora_swiglu.argtypes = [P, I64, ctypes.c_int32, ctypes.c_int32, P, I64, Q, P]
    lib.lora_swiglu_backward.argtypes = [P, I64, P, I64, ctypes.c_int32, ctypes.c_int32, P, I64, Q, P]
    lib.lora_status_string.restype = ctypes.c_char_p
    lib.lora_status_string.argtypes = [ctypes.c_int]
    lib.lora_last_error.restype = ctypes.c_char_p
    lib.lora_version.restype = ctypes.c_int
    for name in EXPORTS:
        if name not in ("lora_status_string", "lora_last_error", "lora_version"):
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int):
    if status != LORA_OK:
        lib = load()
        raise LoraError(status, lib.lora_last_error().decode())


def _ptr(t) -> int:
    """Device or host address of a torch tensor / numpy array (0 for None)."""
    if t is None:
        return 0
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream_handle(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Adapters:
    """Adapters resident on the GPU: device pointer tables + host ranks/scales.

    A, B: sequences of device bf16 tensors, A[i] [r_i, h_in], B[i] [h_out, r_i]
    (None allowed for rank 0). The pointer tables are int64 device tensors,
    so they can be rewritten in place between calls. With host_tables (the
    default) host copies of the tables go with every call too, and small
    launches take the addresses from them: after rewriting a device table in
    place, rewrite A_host / B_host (uint64 numpy arrays) the same way, or
    build the object with host_tables=False.
    """

    def __init__(self, A: Sequence, B: Sequence, ranks, scales, h_in: int, h_out: int,
                 device=None, host_tables: bool = True):
        import torch
        self.A, self.B = list(A), list(B)
        self.ranks = np.ascontiguousarray(ranks, dtype=np.int32)
        self.scales = np.ascontiguousarray(scales, dtype=np.float32)
        self.h_in, self.h_out = int(h_in), int(h_out)
        dev = device if device is not None else "cuda"
        self.A_ptrs = torch.tensor([_ptr(a) for a in self.A], dtype=torch.int64, device=dev)
        self.B_ptrs = torch.tensor([_ptr(b) for b in self.B], dtype=torch.int64, device=dev)
        self.A_host = np.array([_ptr(a) for a in self.A], dtype=np.uint64)
        self.B_host = np.array([_ptr(b) for b in self.B], dtype=np.uint64)
        self._c = CAdapters(len(self.ranks), self.h_in, self.h_out, _ptr(self.A_ptrs),
                            _ptr(self.B_ptrs), self.ranks.ctypes.data, self.scales.ctypes.data,
                            self.A_host.ctypes.data if host_tables else 0,
                            self.B_host.ctypes.data if host_tables else 0)

    @property
    def c(self):
        return ctypes.byref(self._c)


class Segments:
    """A batch in sorted-position order cut into one-adapter segments.

    seg_starts [S+1] and seg_adapter [S] are host arrays; token_rows is an
    optional int32 device tensor (row of x/y used by each sorted position);
    token_rows_host an optional int32 host array with the same rows (small
    forward launches carry it in their arguments; token_rows may then be
    None for them).
    """

    def __init__(self, seg_starts, seg_adapter, token_rows=None, token_rows_host=None):
        self.seg_starts = np.ascontiguousarray(seg_starts, dtype=np.int32)
        self.seg_adapter = np.ascontiguousarray(seg_adapter, dtype=np.int32)
        self.token_rows = token_rows
        S = int(self.seg_adapter.shape[0])
        T = int(self.seg_starts[-1]) if self.seg_starts.size else 0
        self.token_rows_host = None
        if token_rows_host is not None:
            self.token_rows_host = np.ascontiguousarray(token_rows_host, dtype=np.int32)
            if self.token_rows_host.shape != (T,):
                raise ValueError(f"token_rows_host must hold {T} rows, got shape {self.token_rows_host.shape}")
        self._c = CSegments(T, S, self.seg_starts.ctypes.data if S or self.seg_starts.size else 0,
                            self.seg_adapter.ctypes.data if S else 0, _ptr(token_rows),
                            self.token_rows_host.ctypes.data if self.token_rows_host is not None else 0)

    @property
    def num_tokens(self) -> int:
        return int(self._c.num_tokens)

    @property
    def c(self):
        return ctypes.byref(self._c)


def segments_from_ids(ids: np.ndarray, num_adapters: int):
    """Host bookkeeping: (perm [T], seg_starts [N+2], seg_adapter [N+1])."""
    lib = load()
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    T = int(ids.shape[0])
    perm = np.zeros(max(T, 1), np.int32)
    starts = np.zeros(num_adapters + 2, np.int32)
    adap = np.zeros(num_adapters + 1, np.int32)
    _check(lib.lora_segments_from_ids(ids.ctypes.data if T else None, T, int(num_adapters),
                                      perm.ctypes.data, starts.ctypes.data, adap.ctypes.data))
    return perm[:T], starts, adap


def workspace_size(op: int, adapters: Adapters, segments: Optional[Segments] = None) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    _check(lib.lora_workspace_size(op, adapters.c, segments.c if segments is not None else None,
                                   ctypes.byref(n)))
    return int(n.value)


def new_workspace(op: int, adapters: Adapters, segments: Optional[Segments] = None, device="cuda"):
    """A zero-filled workspace tensor of the size `op` needs."""
    import torch
    n = workspace_size(op, adapters, segments)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _ws(ws):
    if ws is None:
        return 0, 0
    return _ptr(ws), int(ws.numel() * ws.element_size())


def sgmv_shrink(x, adapters: Adapters, segments: Segments, u, ws=None, stream=None):
    lib = load()
    wp, wb = _ws(ws)
    _check(lib.lora_sgmv_shrink(_ptr(x), x.stride(0), adapters.c, segments.c, _ptr(u), u.stride(0),
                                wp, wb, _stream_handle(stream)))


def sgmv_expand(u, adapters: Adapters, segments: Segments, y, ws=None, stream=None):
    lib = load()
    wp, wb = _ws(ws)
    _check(lib.lora_sgmv_expand(_ptr(u), u.stride(0), adapters.c, segments.c, _ptr(y), y.stride(0),
                                wp, wb, _stream_handle(stream)))


def sgmv_fused(x, adapters: Adapters, segments: Segments, y, u_save=None, ws=None, stream=None):
    lib = load()
    wp, wb = _ws(ws)
    ldu = u_save.stride(0) if u_save is not None else 0
    _check(lib.lora_sgmv_fused(_ptr(x), x.stride(0), adapters.c, segments.c, _ptr(y), y.stride(0),
                               _ptr(u_save), ldu, wp, wb, _stream_handle(stream)))


def packed_backward(x, dy, u, adapters: Adapters, segments: Segments, dx, dA_ptrs, dB_ptrs,
                    flags: int = 0, ws=None, stream=None):
    """dA_ptrs / dB_ptrs: int64 device tensors of fp32 gradient addresses."""
    lib = load()
    wp, wb = _ws(ws)
    _check(lib.lora_packed_backward(
        _ptr(x), x.stride(0) if x is not None else 0, _ptr(dy), dy.stride(0) if dy is not None else 0,
        _ptr(u), u.stride(0) if u is not None else 0, adapters.c, segments.c, _ptr(dx),
        dx.stride(0) if dx is not None else 0, _ptr(dA_ptrs), _ptr(dB_ptrs), int(flags), wp, wb,
        _stream_handle(stream)))


def sgmv_fused_noalloc(x, adapters: Adapters, segments: Segments, y, u_save=None, stream=None):
    """lora_sgmv_fused_noalloc: the fused call with the library's static
    device scratch instead of a workspace."""
    lib = load()
    ldu = u_save.stride(0) if u_save is not None else 0
    _check(lib.lora_sgmv_fused_noalloc(_ptr(x), x.stride(0), adapters.c, segments.c, _ptr(y), y.stride(0),
                                       _ptr(u_save), ldu, _stream_handle(stream)))


class GraphAdapters:
    """Adapters described only by device tables (for lora_sgmv_fused_graph):
    int64 A/B pointer tables, int32 ranks and float32 scales, all device
    tensors the caller may rewrite between graph replays, plus the host bound
    max_rank."""

    def __init__(self, A_ptrs, B_ptrs, ranks, scales, h_in: int, h_out: int, max_rank: int):
        import torch
        n = int(ranks.numel())
        for name, t, dt in (("A_ptrs", A_ptrs, torch.int64), ("B_ptrs", B_ptrs, torch.int64),
                            ("ranks", ranks, torch.int32), ("scales", scales, torch.float32)):
            if not t.is_cuda or t.dtype != dt or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{name} must be a contiguous {dt} device tensor of {n} entries")
        self.A_ptrs, self.B_ptrs, self.ranks, self.scales = A_ptrs, B_ptrs, ranks, scales
        self.h_in, self.h_out, self.max_rank = int(h_in), int(h_out), int(max_rank)
        self._c = CGraphAdapters(int(ranks.numel()), self.h_in, self.h_out, self.max_rank, _ptr(A_ptrs),
                                 _ptr(B_ptrs), _ptr(ranks), _ptr(scales))

    @property
    def c(self):
        return ctypes.byref(self._c)


def workspace_size_graph(adapters: GraphAdapters, num_tokens: int) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    _check(lib.lora_workspace_size_graph(adapters.c, int(num_tokens), ctypes.byref(n)))
    return int(n.value)


def new_workspace_graph(adapters: GraphAdapters, num_tokens: int, device="cuda"):
    import torch
    return torch.zeros(max(workspace_size_graph(adapters, num_tokens), 256), dtype=torch.uint8, device=device)


def sgmv_fused_graph(x, adapters: GraphAdapters, token_ids, y, ws, stream=None):
    """lora_sgmv_fused_graph: x, y in request order, token_ids an int32 device
    tensor of one adapter id per row of x."""
    import torch
    lib = load()
    T = int(token_ids.numel())
    if not token_ids.is_cuda or token_ids.dtype != torch.int32 or not token_ids.is_contiguous():
        raise ValueError("token_ids must be a contiguous int32 device tensor")
    for name, t, w in (("x", x, adapters.h_in), ("y", y, adapters.h_out)):
        if t.dtype != torch.bfloat16 or t.dim() != 2 or t.shape[0] < T or t.shape[1] != w or t.stride(1) != 1:
            raise ValueError(f"{name} must be a bf16 [>= {T}, {w}] matrix with unit column stride")
    wp, wb = _ws(ws)
    _check(lib.lora_sgmv_fused_graph(_ptr(x), x.stride(0), adapters.c, _ptr(token_ids), int(token_ids.numel()),
                                     _ptr(y), y.stride(0), wp, wb, _stream_handle(stream)))


def _multi_tables(adapters: Sequence[Adapters]):
    """C array of lora_adapters_t pointers (kept alive by the caller)."""
    arr = (ctypes.POINTER(CAdapters) * len(adapters))(*[ctypes.pointer(a._c) for a in adapters])
    return arr


def workspace_size_multi(adapters: Sequence[Adapters], segments: Segments) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    arr = _multi_tables(adapters)
    _check(lib.lora_workspace_size_multi(len(adapters), ctypes.cast(arr, ctypes.c_void_p), segments.c,
                                         ctypes.byref(n)))
    return int(n.value)


def new_workspace_multi(adapters: Sequence[Adapters], segments: Segments, device="cuda"):
    """A zero-filled workspace tensor for sgmv_fused_multi."""
    import torch
    return torch.zeros(max(workspace_size_multi(adapters, segments), 256), dtype=torch.uint8, device=device)


def sgmv_fused_multi(x, adapters: Sequence[Adapters], segments: Segments, ys: Sequence, ws=None, stream=None):
    """One launch for several projections over the same x: ys[p] +=
    s B_p,i (A_p,i x) with projection p's adapters."""
    import torch
    if len(ys) != len(adapters):
        raise ValueError(f"sgmv_fused_multi: {len(adapters)} adapter sets but {len(ys)} outputs")
    for p, y in enumerate(ys):
        if y.dtype != torch.bfloat16 or y.dim() != 2 or y.stride(1) != 1:
            raise ValueError(f"sgmv_fused_multi: ys[{p}] must be a 2-D bfloat16 tensor with unit column stride")
    lib = load()
    wp, wb = _ws(ws)
    arr = _multi_tables(adapters)
    yp = (ctypes.c_void_p * len(ys))(*[_ptr(y) for y in ys])
    ld = (ctypes.c_int64 * len(ys))(*[y.stride(0) for y in ys])
    _check(lib.lora_sgmv_fused_multi(_ptr(x), x.stride(0), len(adapters), ctypes.cast(arr, ctypes.c_void_p),
                                     segments.c, ctypes.cast(yp, ctypes.c_void_p),
                                     ctypes.cast(ld, ctypes.c_void_p), wp, wb, _stream_handle(stream)))


# ---------------------------------------------------------------------------
# 8-bit rows and weights, the frozen projection, the gated activation
# ---------------------------------------------------------------------------
class _Q8:
    """A matrix in 8 bits: e4m3 values [rows, >= 128 * ceil(width / 128)] and
    biased power-of-two exponents, one per 128 columns of `block_rows` rows."""

    block_rows = 1

    def __init__(self, values, exps, width: int, rows: Optional[int] = None):
        import torch
        if (values.dtype not in (torch.uint8, torch.float8_e4m3fn) or values.dim() != 2
                or values.shape[0] > 0 and values.stride(1) != 1):
            raise ValueError("values must be a 2-D uint8 or float8_e4m3fn tensor with unit column stride")
        if exps.dtype != torch.uint8 or exps.dim() != 2 or exps.shape[0] > 0 and exps.stride(1) != 1:
            raise ValueError("exps must be a 2-D uint8 tensor with unit column stride")
        self.rows = int(values.shape[0] if rows is None else rows)
        self.width = int(width)
        blocks, erows = -(-self.width // 128), -(-self.rows // self.block_rows)
        whole = -(-blocks // 4) * 4  # whole dwords of exponents: the products read four blocks at a time
        if self.rows < 0 or self.rows > values.shape[0] or values.shape[1] < 128 * blocks:
            raise ValueError(f"values of shape {tuple(values.shape)} do not hold {self.rows} rows of {128 * blocks} bytes")
        ld, lde = values.stride(0), exps.stride(0)
        # (a row that no other follows may have any stride)
        if self.rows <= 1:
            ld = 128 * blocks
        if erows == 0 or erows == 1 and max(exps.shape[1], lde) >= whole:
            lde = whole
        if exps.shape[0] < erows or lde < whole or exps.shape[1] < blocks:
            raise ValueError(f"exps of shape {tuple(exps.shape)} do not hold {erows} rows of {blocks} blocks "
                             "with a stride that is a multiple of 4")
        if values.device != exps.device:
            raise ValueError(f"values are on {values.device}, exps on {exps.device}")
        self.values, self.exps = values, exps
        self.dev = values.get_device()
        self._c = CQ8(_ptr(values), ld, _ptr(exps), lde, self.rows, self.width,
                      self.block_rows)
        self.addr = ctypes.addressof(self._c)


class Q8Rows(_Q8):
    """8-bit rows (activations, checkpoints): one scale per row and 128 columns."""


class Q8Weights(_Q8):
    """8-bit weights [h_out, h_in]: one scale per 128 x 128 block."""

    block_rows = 128


def _new_q8(cls, rows: int, width: int, device):
    import torch
    blocks, erows = -(-int(width) // 128), -(-int(rows) // cls.block_rows)
    v = torch.empty((int(rows), 128 * blocks), dtype=torch.uint8, device=device)
    e = torch.empty((erows, -(-blocks // 4) * 4), dtype=torch.uint8, device=device)
    return cls(v, e, width)


def new_q8_rows(rows: int, width: int, device="cuda") -> Q8Rows:
    return _new_q8(Q8Rows, rows, width, device)


def new_q8_weights(rows: int, width: int, device="cuda") -> Q8Weights:
    return _new_q8(Q8Weights, rows, width, device)


def _rows_arg(name: str, t, rows: int, width: int, dev: int) -> int:
    """The row stride of a bfloat16 [>= rows, width] tensor on GPU `dev`."""
    if t.dtype is _torch.bfloat16 and t.get_device() == dev:
        shape = t.shape
        if len(shape) == 2 and shape[0] >= rows and shape[1] == width:
            stride, step = t.stride()
            if shape[0] <= 1 and (step == 1 or shape[0] == 0):
                return width  # (a row that no other follows may have any stride)
            if step == 1:
                return stride
    raise ValueError(f"{name} must be a bfloat16 [>= {rows}, {width}] matrix with unit column stride on "
                     f"{_dev_name(dev)}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _q8_arg(name: str, q: _Q8, dev: int) -> int:
    if q.dev != dev:
        raise ValueError(f"{name} is on {_dev_name(q.dev)}, expected {_dev_name(dev)}")
    return q.addr


_INDEX_TYPES, _ADDRESS_TYPES = ("torch.int32",), ("torch.int64", "torch.uint64")


def _largest_rank(adapters: Adapters, segments: Segments) -> int:
    used = segments.seg_adapter[(segments.seg_adapter >= 0) & (segments.seg_adapter < len(adapters.ranks))]
    return int(adapters.ranks[used].max(initial=0))


def _dev_name(dev: int) -> str:
    return f"cuda:{dev}" if dev >= 0 else "cpu"


def _call_on(dev: int, stream, fn, *args):
    """Calls fn(*args, stream) with GPU `dev` current, on `stream` or that
    GPU's current stream. (A decode step makes many such calls and each is a
    few microseconds of GPU work, so the host's share is kept small.)"""
    if dev < 0:
        raise ValueError("device tensors are needed, got cpu")
    if stream is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    cuda = _torch._C
    if dev != cuda._cuda_getDevice():
        with _torch.cuda.device(dev):
            return _call_on(dev, stream, fn, *args)
    st = fn(*args, cuda._cuda_getCurrentRawStream(dev) if stream is None else _stream_handle(stream))
    if st:
        _check(st)


def q8_quantize(x, out: _Q8, out_t: Optional[Q8Weights] = None, stream=None):
    """Stores bf16 x in 8 bits (Q8Rows or Q8Weights); with out_t the
    transposed weights too."""
    lib, dev = _lib or load(), out.dev
    ldx = _rows_arg("x", x, out.rows, out.width, dev)
    ot = _q8_arg("out_t", out_t, dev) if out_t is not None else None
    _call_on(dev, stream, lib.lora_q8_quantize, x.data_ptr(), ldx, out.addr, ot)


def q8_dequantize(q: _Q8, x, stream=None):
    """Restores an 8-bit matrix to bf16 x."""
    lib = _lib or load()
    ldx = _rows_arg("x", x, q.rows, q.width, q.dev)
    _call_on(q.dev, stream, lib.lora_q8_dequantize, q.addr, x.data_ptr(), ldx)


def q8_matmul(x: Q8Rows, w: Q8Weights, y, accumulate: bool = False, stream=None):
    """y = x w^T (or y += x w^T) on 8-bit operands; y bf16 [x.rows, w.rows]."""
    lib, dev = _lib or load(), x.dev
    ldy = _rows_arg("y", y, x.rows, w.rows, dev)
    _call_on(dev, stream, lib.lora_q8_matmul, x.addr, _q8_arg("w", w, dev), y.data_ptr(), ldy,
             1 if accumulate else 0)


def packed_backward_q8(x: Q8Rows, dy, u, adapters: Adapters, segments: Segments, dx, dA_ptrs, dB_ptrs,
                       flags: int = 0, ws=None, stream=None):
    """packed_backward with x as the 8-bit checkpoint; u (the forward's
    u_save) is required."""
    lib, T, dev = _lib or load(), segments.num_tokens, x.dev
    lddy = _rows_arg("dy", dy, T, adapters.h_out, dev)
    lddx = _rows_arg("dx", dx, T, adapters.h_in, dev) if dx is not None else 0
    ldu = 0
    if u is not None and u.dim() == 2:
        ldu = u.stride(0) if u.shape[0] > 1 else u.shape[1]
    # (rows that follow each other are as wide as their stride, which the call checks)
    if (u is None or u.get_device() != dev or u.dtype is not _torch.float32 or u.dim() != 2 or u.shape[0] < T
            or u.shape[0] > 0 and u.stride(1) != 1 or u.shape[1] != ldu and u.shape[1] < _largest_rank(adapters, segments)):
        raise ValueError(f"u must be a float32 [>= {T}, >= largest rank] matrix with unit column stride on {_dev_name(dev)}")
    for name, t in (("adapters", adapters.A_ptrs), ("token_rows", segments.token_rows), ("dA_ptrs", dA_ptrs),
                    ("dB_ptrs", dB_ptrs), ("ws", ws)):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected {_dev_name(dev)}")
    # tables that the kernels index: a shorter or narrower one would be read behind its end
    for name, t, n, types in (("token_rows", segments.token_rows, T, _INDEX_TYPES),
                              ("dA_ptrs", dA_ptrs, len(adapters.ranks), _ADDRESS_TYPES),
                              ("dB_ptrs", dB_ptrs, len(adapters.ranks), _ADDRESS_TYPES)):
        if t is not None and (str(t.dtype) not in types or t.numel() < n or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {types[0]} tensor of {n} entries, got {t.dtype} {tuple(t.shape)}")
    wp, wb = _ws(ws)
    _call_on(dev, stream, lib.lora_packed_backward_q8, x.addr, dy.data_ptr(), lddy, u.data_ptr(), ldu,
             adapters.c, segments.c, _ptr(dx), lddx, _ptr(dA_ptrs), _ptr(dB_ptrs), int(flags), wp, wb)


def swiglu(gate_up, h=None, hq: Optional[Q8Rows] = None, stream=None):
    """h = silu(gate) * up of gate_up [T, 2F], as bf16 rows and/or 8-bit rows."""
    lib, dev = _lib or load(), gate_up.get_device()
    T, W = gate_up.shape
    F = W // 2
    ld = _rows_arg("gate_up", gate_up, T, 2 * F, dev)
    ldh = _rows_arg("h", h, T, F, dev) if h is not None else 0
    q = _q8_arg("hq", hq, dev) if hq is not None else None
    _call_on(dev, stream, lib.lora_swiglu, gate_up.data_ptr(), ld, T, F, _ptr(h), ldh, q)


def swiglu_backward(gate_up, dh, dgate_up=None, dgate_up_q: Optional[Q8Rows] = None, stream=None):
    """The gradient of swiglu's input, [T, 2F], as bf16 rows and/or 8-bit rows."""
    lib, dev = _lib or load(), gate_up.get_device()
    T, W = gate_up.shape
    F = W // 2
    ld = _rows_arg("gate_up", gate_up, T, 2 * F, dev)
    lddh = _rows_arg("dh", dh, T, F, dev)
    ldd = _rows_arg("dgate_up", dgate_up, T, 2 * F, dev) if dgate_up is not None else 0
    q = _q8_arg("dgate_up_q", dgate_up_q, dev) if dgate_up_q is not None else None
    _call_on(dev, stream, lib.lora_swiglu_backward, gate_up.data_ptr(), ld, dh.data_ptr(), lddh, T, F,
             _ptr(dgate_up), ldd, q)


class CPlanItem(ctypes.Structure):
    """lora_plan_item_t of the internal inspection entry (csrc/lora_inspect.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("launch", "phase", "block", "grid", "mode", "kind", "tile", "adapter", "proj", "rank",
                 "tok0", "ntok", "lo", "hi", "part", "aux")]


INSPECT_WITH_U, INSPECT_WITH_DX, INSPECT_ACCUMULATE = 1, 2, 4
PHASE_FWD, PHASE_WGRAD, PHASE_REDUCE, PHASE_TRANSPOSE, PHASE_PLAN = 0, 1, 2, 3, 4


def inspect_plan(op: int, adapters, segments: Segments, options: int = 0, cus: int = 256, xccs: int = 8):
    """Host-only listing of every workgroup the call `op` would launch
    (no GPU involved). adapters: one Adapters-like object, or a sequence of
    them for a multi-projection fused call. Returns (items, ranges): a numpy
    structured array with the lora_plan_item_t fields, and an int32 [n, 2]
    array of (first position, count) token ranges of weight-gradient jobs."""
    lib = load()
    fn = lib.lora_inspect_plan
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int, ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(CSegments), ctypes.c_uint32,
                   ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                   ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p, ctypes.c_int64,
                   ctypes.POINTER(ctypes.c_int64)]
    ads = list(adapters) if isinstance(adapters, (list, tuple)) else [adapters]
    arr = _multi_tables(ads)
    n_items = ctypes.c_int64(0)
    n_ranges = ctypes.c_int64(0)
    cap, rcap = 1 << 14, 1 << 12
    while True:
        items = (CPlanItem * cap)()
        ranges = (ctypes.c_int32 * (2 * rcap))()
        _check(fn(op, len(ads), ctypes.cast(arr, ctypes.c_void_p), segments.c, options, cus, xccs,
                  ctypes.cast(items, ctypes.c_void_p), cap, ctypes.byref(n_items),
                  ctypes.cast(ranges, ctypes.c_void_p), rcap, ctypes.byref(n_ranges)))
        if n_items.value <= cap and n_ranges.value <= rcap:
            break
        cap = max(cap, int(n_items.value))
        rcap = max(rcap, int(n_ranges.value))
    dt = np.dtype([(f, np.int32) for f, _ in CPlanItem._fields_])
    out = np.frombuffer(bytes(items), dtype=dt, count=int(n_items.value)).copy()
    rg = np.frombuffer(bytes(ranges), dtype=np.int32, count=2 * int(n_ranges.value)).reshape(-1, 2).copy()
    return out, rg


def inspect_graph(num_adapters: int, h_in: int, h_out: int, max_rank: int, num_tokens: int, tiles: int,
                  cus: int = 256, xccs: int = 8):
    """Host-only listing of the workgroups of a device-planned call over
    num_tokens ids whose batch turns out to have `tiles` tiles (stand-in
    device tables, never dereferenced). Returns a numpy structured array with
    the lora_plan_item_t fields."""
    lib = load()
    fn = lib.lora_inspect_graph
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(CGraphAdapters), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                   ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    fake = 1 << 40
    ga = CGraphAdapters(int(num_adapters), int(h_in), int(h_out), int(max_rank), fake, fake + 4096, fake + 8192,
                        fake + 12288)
    n = ctypes.c_int64(0)
    cap = 1 << 12
    while True:
        items = (CPlanItem * cap)()
        _check(fn(ctypes.byref(ga), int(num_tokens), int(tiles), int(cus), int(xccs), ctypes.cast(items, ctypes.c_void_p),
                  cap, ctypes.byref(n)))
        if n.value <= cap:
            break
        cap = int(n.value)
    dt = np.dtype([(f, np.int32) for f, _ in CPlanItem._fields_])
    return np.frombuffer(bytes(items), dtype=dt, count=int(n.value)).copy()


class CMatmulKernel(ctypes.Structure):
    """lora_matmul_kernel_t of the internal inspection entry (csrc/lora_inspect.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("kernels", "kernel", "tokens", "columns", "groups", "stages", "blocks", "exps")]


def inspect_matmul(num_tokens: int, width: int, h_out: int) -> CMatmulKernel:
    """Host-only: the kernel that q8_matmul launches for these sizes."""
    lib = load()
    fn = lib.lora_inspect_matmul
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(CMatmulKernel)]
    out = CMatmulKernel()
    _check(fn(int(num_tokens), int(width), int(h_out), ctypes.byref(out)))
    return out


def version() -> int:
    return int(load().lora_version())
