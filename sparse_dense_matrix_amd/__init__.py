"""Python binding of libspmm.so: sparse x dense matrix multiplication on
MI355X (gfx950).

The functions carry the C ABI's names (include/spmm.h) and only marshal
arguments: packing runs in the library's host code and every multiplication
step runs in its HIP kernels.  PyTorch is used for device memory and streams
only (spmm_execute takes torch tensors or raw device pointers).

There is no fallback: if libspmm.so is missing or fails to load, importing
this package raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import numpy as np

__all__ = [
    "SpmmError", "Matrix", "Plan", "F32", "BF16", "I8", "I32", "F16",
    "FORMAT_BCSR", "FORMAT_WCSR", "FORMAT_24", "FORMAT_TVW", "FORMAT_SLIDE", "FORMAT_ATTN", "FORMAT_ROPE",
    "ARRAY_ROW_PTR", "ARRAY_COL_IDX", "ARRAY_VALS", "ARRAY_META",
    "ARRAY_CHUNK_WINDOW", "ARRAY_CHUNK_BEGIN", "ARRAY_ROW_PERM", "ARRAY_COL_PERM",
    "spmm_pack_bcsr", "spmm_pack_bcsr_csr", "spmm_pack_wcsr", "spmm_pack_24", "spmm_pack_tvw", "spmm_pack_slide",
    "spmm_matrix_info",
    "spmm_matrix_array", "spmm_plan", "spmm_plan_info", "spmm_execute", "spmm_execute_noalloc",
    "spmm_plan_sddmm", "spmm_execute_sddmm",
    "spmm_plan_attn", "spmm_execute_attn_pool", "spmm_execute_attn_select", "spmm_execute_attn",
    "spmm_execute_attn_backward", "spmm_execute_attn_cache",
    "spmm_execute_attn_write", "spmm_execute_attn_read", "spmm_execute_attn_pool8", "spmm_execute_attn_cache8",
    "spmm_plan_attn_rope", "spmm_execute_attn_rope", "spmm_execute_attn_rope_backward",
    "spmm_status_str", "spmm_last_error", "LIB_PATH", "EXPORTS",
]

HERE = os.path.dirname(os.path.abspath(__file__))
# SPMM_LIBRARY may point at another build of the same library
LIB_PATH = os.environ.get("SPMM_LIBRARY") or os.path.join(HERE, "libspmm.so")

F32, BF16, I8, I32, F16 = 0, 1, 2, 3, 4
_ELEM = {F32: 4, BF16: 2, I8: 1, I32: 4}  # bytes per element of each type
FORMAT_BCSR, FORMAT_WCSR, FORMAT_24, FORMAT_TVW, FORMAT_SLIDE, FORMAT_ATTN, FORMAT_ROPE = 0, 1, 2, 3, 4, 5, 6
(ARRAY_ROW_PTR, ARRAY_COL_IDX, ARRAY_VALS, ARRAY_META, ARRAY_CHUNK_WINDOW,
 ARRAY_CHUNK_BEGIN, ARRAY_ROW_PERM, ARRAY_COL_PERM) = range(8)

# Default row-window shape for WCSR: 0 lets the library choose (W rows per
# window, at most T stored entries per chunk; one wavefront reduces one chunk).
DEFAULT_WINDOW_ROWS = 0
DEFAULT_MAX_CHUNK_NNZ = 0

# every symbol include/spmm.h declares
EXPORTS = (
    "spmm_pack_bcsr", "spmm_pack_bcsr_csr", "spmm_pack_wcsr", "spmm_pack_24", "spmm_pack_tvw", "spmm_pack_slide",
    "spmm_matrix_info",
    "spmm_matrix_array", "spmm_matrix_destroy", "spmm_plan", "spmm_plan_info",
    "spmm_plan_destroy", "spmm_execute", "spmm_execute_noalloc", "spmm_plan_sddmm",
    "spmm_execute_sddmm",
    "spmm_plan_attn", "spmm_execute_attn_pool", "spmm_execute_attn_select", "spmm_execute_attn",
    "spmm_execute_attn_backward", "spmm_execute_attn_cache",
    "spmm_execute_attn_write", "spmm_execute_attn_read", "spmm_execute_attn_pool8", "spmm_execute_attn_cache8",
    "spmm_plan_attn_rope", "spmm_execute_attn_rope", "spmm_execute_attn_rope_backward",
    "spmm_status_str", "spmm_last_error",
)


class MatrixInfo(C.Structure):
    _fields_ = [("format", C.c_int32), ("dtype", C.c_int32), ("m", C.c_int64),
                ("k", C.c_int64), ("nnz", C.c_int64), ("nnzb", C.c_int64),
                ("block_m", C.c_int32), ("block_k", C.c_int32),
                ("window_rows", C.c_int32), ("max_chunk_nnz", C.c_int64),
                ("num_windows", C.c_int64), ("num_chunks", C.c_int64)]


class PlanInfo(C.Structure):
    _fields_ = [("format", C.c_int32), ("device", C.c_int32), ("m", C.c_int64),
                ("k", C.c_int64), ("n", C.c_int64), ("device_bytes", C.c_int64),
                ("workspace_bytes", C.c_int64), ("num_split_rows", C.c_int64),
                ("num_slots", C.c_int64), ("tile_m", C.c_int32), ("tile_n", C.c_int32),
                ("grid", C.c_int64)]


class AttnDesc(C.Structure):
    _fields_ = [("batch", C.c_int64), ("queries", C.c_int64), ("keys", C.c_int64),
                ("heads_q", C.c_int32), ("heads_kv", C.c_int32), ("dim", C.c_int32),
                ("dtype", C.c_int32), ("q_block", C.c_int32), ("max_blocks", C.c_int32),
                ("sink_blocks", C.c_int32), ("local_blocks", C.c_int32), ("backward", C.c_int32),
                ("scale", C.c_float)]


class RopeDesc(C.Structure):
    _fields_ = [("batch", C.c_int64), ("tokens", C.c_int64), ("heads_q", C.c_int32), ("heads_kv", C.c_int32),
                ("dim", C.c_int32), ("dtype", C.c_int32), ("pairs", C.c_int32), ("axes", C.c_int32),
                ("interleaved", C.c_int32), ("backward", C.c_int32), ("eps", C.c_float),
                ("freqs", C.c_void_p), ("axis", C.c_void_p)]


def _load():
    # One HIP runtime per process: torch ships its own libamdhip64 with the
    # same soname as the system one libspmm.so links.  Loading torch first
    # makes libspmm.so bind to that already-loaded runtime; two runtimes in
    # one process do not share devices.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built (run __graft_entry__.build() or "
                          f"python sparse_dense_matrix_amd/build.py)")
    L = C.CDLL(LIB_PATH)
    P, i64, i32, st = C.c_void_p, C.c_int64, C.c_int32, C.c_int
    sig = {
        "spmm_pack_bcsr": (st, [i64, i64, i32, i32, st, P, i64, C.POINTER(P)]),
        "spmm_pack_wcsr": (st, [i64, i64, st, P, P, P, i32, i64, C.POINTER(P)]),
        "spmm_pack_bcsr_csr": (st, [i64, i64, st, P, P, P, i32, i32, i32, C.POINTER(P)]),
        "spmm_pack_24": (st, [i64, i64, i32, P, i64, C.POINTER(P)]),
        "spmm_pack_tvw": (st, [i64, i64, i32, P, i64, i32, i32, C.POINTER(P)]),
        "spmm_pack_slide": (st, [i64, i64, P, i64, i32, C.POINTER(P)]),
        "spmm_matrix_info": (st, [P, C.POINTER(MatrixInfo)]),
        "spmm_matrix_array": (st, [P, i32, C.POINTER(P), C.POINTER(i64)]),
        "spmm_matrix_destroy": (None, [P]),
        "spmm_plan": (st, [P, i64, st, st, i32, C.POINTER(P)]),
        "spmm_plan_info": (st, [P, C.POINTER(PlanInfo)]),
        "spmm_plan_destroy": (None, [P]),
        "spmm_execute": (st, [P, P, i64, P, i64, P]),
        "spmm_execute_noalloc": (st, [P, P, i64, P, i64, P]),
        "spmm_plan_sddmm": (st, [P, i64, st, i32, C.POINTER(P)]),
        "spmm_execute_sddmm": (st, [P, P, i64, P, i64, P, P]),
        "spmm_plan_attn": (st, [C.POINTER(AttnDesc), i32, C.POINTER(P)]),
        "spmm_execute_attn_pool": (st, [P, P, i64, P, P, P, P, P, P]),
        "spmm_execute_attn_select": (st, [P, P, P, P, i64, P, P, P, P, P]),
        "spmm_execute_attn": (st, [P] * 10),
        "spmm_execute_attn_backward": (st, [P] * 14),
        "spmm_execute_attn_cache": (st, [P, P, P, P, i64] + [P] * 8),
        "spmm_execute_attn_write": (st, [P] * 7 + [i64] + [P] * 4),
        "spmm_execute_attn_read": (st, [P] * 5 + [i64] + [P] * 5),
        "spmm_execute_attn_pool8": (st, [P] * 3 + [i64] + [P] * 6),
        "spmm_execute_attn_cache8": (st, [P] * 6 + [i64] + [P] * 8),
        "spmm_plan_attn_rope": (st, [C.POINTER(RopeDesc), i32, C.POINTER(P)]),
        "spmm_execute_attn_rope": (st, [P] * 11),
        "spmm_execute_attn_rope_backward": (st, [P] * 15),
        "spmm_status_str": (C.c_char_p, [st]),
        "spmm_last_error": (C.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


_lib = _load()


def lib():
    return _lib


class SpmmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        self.name = spmm_status_str(status)
        self.message = spmm_last_error()
        super().__init__(f"{where}: {self.name}: {self.message}")


def spmm_status_str(status: int) -> str:
    return _lib.spmm_status_str(status).decode()


def spmm_last_error() -> str:
    return _lib.spmm_last_error().decode()


def _check(status: int, where: str):
    if status != 0:
        raise SpmmError(status, where)


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(C.c_void_p)


class Matrix:
    """Owns one reference to a packed sparse operand."""

    def __init__(self, handle):
        self.handle = handle

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.spmm_matrix_destroy(h)

    def info(self) -> dict:
        return spmm_matrix_info(self)


class Plan:
    """Owns a device plan (and through it a reference to its matrix).

    `expect` maps each dense operand of an execute call to (rows, cols,
    bytes per element), or ("count", n, bytes) for the SDDMM output, plus
    "device"; torch tensors handed to execute are checked against it so that
    a kernel never reads or writes past them."""

    def __init__(self, handle, expect=None):
        self.handle = handle
        self.expect = expect or {}

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.spmm_plan_destroy(h)

    def info(self) -> dict:
        return spmm_plan_info(self)


def spmm_pack_bcsr(a_bits: np.ndarray, block_m: int = 64, block_k: int = 64,
                   dtype: int = BF16) -> Matrix:
    """BCSR from a dense row-major bf16 matrix given as uint16 bit patterns."""
    a = np.ascontiguousarray(a_bits)
    if a.ndim != 2:
        raise ValueError("a must be 2-D")
    h = C.c_void_p()
    _check(_lib.spmm_pack_bcsr(a.shape[0], a.shape[1], block_m, block_k, dtype, _ptr(a),
                               a.shape[1], C.byref(h)), "spmm_pack_bcsr")
    return Matrix(h)


def spmm_pack_slide(a: np.ndarray, group: int = 8) -> Matrix:
    """(group-2):group weights (group = 2N) as N-1 overlapping 2:4 windows per
    group, from a dense int8 matrix."""
    a = np.ascontiguousarray(a, dtype=np.int8)
    if a.ndim != 2:
        raise ValueError("a must be 2-D")
    h = C.c_void_p()
    _check(_lib.spmm_pack_slide(a.shape[0], a.shape[1], _ptr(a), a.shape[1], group, C.byref(h)),
           "spmm_pack_slide")
    return Matrix(h)


def spmm_pack_tvw(a: np.ndarray, tile_m: int = 256, tile_k: int = 128) -> Matrix:
    """Tile-vector-wise from a dense matrix: int8, or bf16 given as uint16
    bit patterns.  Tiles with a nonzero are stored, 2:4-pruned along k."""
    a = np.asarray(a)
    if a.dtype == np.uint16:
        dtype = BF16
    elif a.dtype == np.int8:
        dtype = I8
    else:
        raise TypeError("spmm_pack_tvw takes int8 or uint16 (bf16 bits) values")
    a = np.ascontiguousarray(a)
    if a.ndim != 2:
        raise ValueError("a must be 2-D")
    h = C.c_void_p()
    _check(_lib.spmm_pack_tvw(a.shape[0], a.shape[1], dtype, _ptr(a), a.shape[1], tile_m, tile_k,
                              C.byref(h)), "spmm_pack_tvw")
    return Matrix(h)


def spmm_pack_bcsr_csr(m: int, k: int, row_ptr, col_idx, vals_bits, reorder: bool = False,
                       block_m: int = 64, block_k: int = 64, dtype: int = BF16) -> Matrix:
    """BCSR from a canonical CSR with bf16 values (uint16 bit patterns),
    optionally after the row/column permutation that clusters entries into
    fewer blocks (read back with ARRAY_ROW_PERM / ARRAY_COL_PERM)."""
    rp = np.ascontiguousarray(row_ptr, dtype=np.int64)
    ci = np.ascontiguousarray(col_idx, dtype=np.int32)
    v = np.ascontiguousarray(vals_bits, dtype=np.uint16)
    if len(rp) != m + 1:
        raise ValueError("row_ptr must have m + 1 entries")
    h = C.c_void_p()
    _check(_lib.spmm_pack_bcsr_csr(m, k, dtype, _ptr(rp), _ptr(ci), _ptr(v), block_m, block_k,
                                   int(bool(reorder)), C.byref(h)), "spmm_pack_bcsr_csr")
    return Matrix(h)


def spmm_pack_wcsr(m: int, k: int, row_ptr, col_idx, vals,
                   window_rows: int = DEFAULT_WINDOW_ROWS,
                   max_chunk_nnz: int = DEFAULT_MAX_CHUNK_NNZ, dtype: int = F32) -> Matrix:
    rp = np.ascontiguousarray(row_ptr, dtype=np.int64)
    ci = np.ascontiguousarray(col_idx, dtype=np.int32)
    v = np.ascontiguousarray(vals, dtype=np.float32)
    if len(rp) != m + 1:
        raise ValueError("row_ptr must have m + 1 entries")
    h = C.c_void_p()
    _check(_lib.spmm_pack_wcsr(m, k, dtype, _ptr(rp), _ptr(ci), _ptr(v), window_rows,
                               max_chunk_nnz, C.byref(h)), "spmm_pack_wcsr")
    return Matrix(h)


def spmm_pack_24(a: np.ndarray) -> Matrix:
    """2:4 from a dense matrix: int8, or bf16 given as uint16 bit patterns."""
    a = np.asarray(a)
    if a.dtype == np.uint16:
        dtype = BF16
    elif a.dtype == np.int8:
        dtype = I8
    else:
        raise TypeError("spmm_pack_24 takes int8 or uint16 (bf16 bits) values")
    a = np.ascontiguousarray(a)
    if a.ndim != 2:
        raise ValueError("a must be 2-D")
    h = C.c_void_p()
    _check(_lib.spmm_pack_24(a.shape[0], a.shape[1], dtype, _ptr(a), a.shape[1], C.byref(h)),
           "spmm_pack_24")
    return Matrix(h)


def spmm_matrix_info(mat: Matrix) -> dict:
    info = MatrixInfo()
    _check(_lib.spmm_matrix_info(mat.handle, C.byref(info)), "spmm_matrix_info")
    return {f: getattr(info, f) for f, _ in MatrixInfo._fields_}


_ARRAY_DTYPES = {
    (FORMAT_BCSR, ARRAY_ROW_PTR): np.int32, (FORMAT_BCSR, ARRAY_COL_IDX): np.int32,
    (FORMAT_BCSR, ARRAY_VALS): np.uint16, (FORMAT_BCSR, ARRAY_ROW_PERM): np.int32,
    (FORMAT_BCSR, ARRAY_COL_PERM): np.int32,
    (FORMAT_WCSR, ARRAY_ROW_PTR): np.int64, (FORMAT_WCSR, ARRAY_COL_IDX): np.int32,
    (FORMAT_WCSR, ARRAY_VALS): np.float32, (FORMAT_WCSR, ARRAY_CHUNK_WINDOW): np.int32,
    (FORMAT_WCSR, ARRAY_CHUNK_BEGIN): np.int64,
    (FORMAT_24, ARRAY_VALS): np.int8, (FORMAT_24, ARRAY_META): np.uint8,
    (FORMAT_TVW, ARRAY_ROW_PTR): np.int32, (FORMAT_TVW, ARRAY_COL_IDX): np.int32,
    (FORMAT_TVW, ARRAY_VALS): np.int8, (FORMAT_TVW, ARRAY_META): np.uint8,
    (FORMAT_SLIDE, ARRAY_VALS): np.int8, (FORMAT_SLIDE, ARRAY_META): np.uint8,
}


def spmm_matrix_array(mat: Matrix, which: int) -> np.ndarray:
    """Copy of a canonical array (see include/spmm.h)."""
    data, count = C.c_void_p(), C.c_int64()
    _check(_lib.spmm_matrix_array(mat.handle, which, C.byref(data), C.byref(count)),
           "spmm_matrix_array")
    info = spmm_matrix_info(mat)
    fmt = info["format"]
    dt = np.dtype(_ARRAY_DTYPES[(fmt, which)])
    if fmt in (FORMAT_TVW, FORMAT_24) and which == ARRAY_VALS and info["dtype"] == BF16:
        dt = np.dtype(np.uint16)
    if count.value == 0:
        return np.zeros(0, dtype=dt)
    buf = (C.c_char * (count.value * dt.itemsize)).from_address(data.value)
    return np.frombuffer(buf, dtype=dt).copy()


def spmm_plan(mat: Matrix, n: int, b_dtype: int, c_dtype: int, device: int = 0) -> Plan:
    h = C.c_void_p()
    _check(_lib.spmm_plan(mat.handle, n, b_dtype, c_dtype, device, C.byref(h)), "spmm_plan")
    mi = spmm_matrix_info(mat)
    return Plan(h, {"b": (mi["k"], n, _ELEM[b_dtype]), "c": (mi["m"], n, _ELEM[c_dtype]),
                    "device": device})


def spmm_plan_info(plan: Plan) -> dict:
    info = PlanInfo()
    _check(_lib.spmm_plan_info(plan.handle, C.byref(info)), "spmm_plan_info")
    return {f: getattr(info, f) for f, _ in PlanInfo._fields_}


def _dev_ptr_ld(t):
    """(pointer, leading dimension) of a 2-D row-major torch tensor.  A tensor
    with no columns has no meaningful strides: its leading dimension is 0."""
    if t.dim() == 2 and t.shape[1] == 0:
        return t.data_ptr(), 0
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("dense operands must be 2-D row-major (stride(1) == 1)")
    return t.data_ptr(), t.stride(0)


def _check_tensor(plan: Plan, name: str, t):
    """Shape, element size and device of a torch tensor against the plan."""
    want = plan.expect.get(name)
    if want is None:
        return
    dev = plan.expect["device"]
    if not t.is_cuda or (t.device.index if t.device.index is not None else 0) != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    rows, cols, elem = want
    if t.element_size() != elem:
        raise ValueError(f"{name} has {t.element_size()}-byte elements; the plan takes {elem}")
    if rows == "count":
        if t.numel() < cols or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with at least {cols} elements")
    elif tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the plan takes ({rows}, {cols})")


def _execute(fn: str, plan: Plan, b, c, stream, ldb, ldc):
    if isinstance(b, int) or isinstance(c, int):
        bp, cp = int(b), int(c)
        if ldb is None or ldc is None:
            raise ValueError("raw pointers need ldb and ldc")
    else:
        _check_tensor(plan, "b", b)
        _check_tensor(plan, "c", c)
        bp, ldb = _dev_ptr_ld(b)
        cp, ldc = _dev_ptr_ld(c)
    if stream is None:
        import torch
        dev = c.device if hasattr(c, "device") else None
        stream = torch.cuda.current_stream(dev).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    _check(getattr(_lib, fn)(plan.handle, C.c_void_p(bp), ldb, C.c_void_p(cp), ldc,
                             C.c_void_p(stream)), fn)


def spmm_execute(plan: Plan, b, c, stream=None, ldb: int | None = None,
                 ldc: int | None = None):
    """C = A * B on `stream` (default: torch's current stream on C's device).

    b and c are torch tensors on the plan's device, or raw device pointers
    with ldb / ldc given."""
    _execute("spmm_execute", plan, b, c, stream, ldb, ldc)


def spmm_execute_noalloc(plan: Plan, b, c, stream=None, ldb: int | None = None,
                         ldc: int | None = None):
    """spmm_execute that allocates nothing: a WCSR plan's partial rows live in
    the library's fixed per-GPU scratch array (calls that overlap on one GPU
    race).  Arguments as for spmm_execute."""
    _execute("spmm_execute_noalloc", plan, b, c, stream, ldb, ldc)


def spmm_plan_sddmm(mat: Matrix, kd: int, dtype: int = F32, device: int = 0) -> Plan:
    """Plan the sampled product out[p] = X[i] . Y[j] over the stored entries
    (i, j) of a WCSR (dtype F32, BF16 or I8) or 64 x 64 BCSR (BF16 or I8)
    matrix, inner dimension kd."""
    h = C.c_void_p()
    _check(_lib.spmm_plan_sddmm(mat.handle, kd, dtype, device, C.byref(h)), "spmm_plan_sddmm")
    mi = spmm_matrix_info(mat)
    count = mi["nnzb"] * 64 * 64 if mi["format"] == 0 else mi["nnz"]
    out_elem = {F32: 4, BF16: 2, I8: 4}[dtype]
    return Plan(h, {"x": (mi["m"], kd, _ELEM[dtype]), "y": (mi["k"], kd, _ELEM[dtype]),
                    "out": ("count", count, out_elem), "device": device})


def spmm_execute_sddmm(plan: Plan, x, y, out, stream=None, ldx: int | None = None,
                       ldy: int | None = None):
    """out[p] for every stored entry on `stream` (default: torch's current
    stream).  x [m, kd] and y [k, kd] are 2-D row-major torch tensors (or raw
    device pointers with ldx / ldy); out (tensor or raw pointer) holds the
    plan's output type: fp32, bf16 bits or int32, one per stored entry (WCSR)
    or [nnzb, 64, 64] (BCSR)."""
    if isinstance(x, int) or isinstance(y, int):
        xp, yp = int(x), int(y)
        if ldx is None or ldy is None:
            raise ValueError("raw pointers need ldx and ldy")
    else:
        _check_tensor(plan, "x", x)
        _check_tensor(plan, "y", y)
        xp, ldx = _dev_ptr_ld(x)
        yp, ldy = _dev_ptr_ld(y)
    if not isinstance(out, int):
        _check_tensor(plan, "out", out)
    op = int(out) if isinstance(out, int) else out.data_ptr()
    if stream is None:
        import torch
        dev = out.device if hasattr(out, "device") else None
        stream = torch.cuda.current_stream(dev).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    _check(_lib.spmm_execute_sddmm(plan.handle, C.c_void_p(xp), ldx, C.c_void_p(yp), ldy,
                                   C.c_void_p(op), C.c_void_p(stream)), "spmm_execute_sddmm")


def spmm_plan_attn(batch: int, queries: int, keys: int, heads_q: int, heads_kv: int, dim: int,
                   dtype: int = BF16, q_block: int = 64, max_blocks: int = 16, sink_blocks: int = 1,
                   local_blocks: int = 1, scale: float | None = None, backward: bool = False,
                   device: int = 0) -> Plan:
    """Plan block-sparse attention of `batch` sequences of `queries` queries
    over at most `keys` keys, in blocks of 64 keys; one list of max_blocks
    blocks for each q_block queries and key head.  dtype is BF16 or F16,
    scale defaults to 1 / sqrt(dim).  With a cache, keys is the table's width
    times 64."""
    if scale is not None and not scale > 0:
        raise ValueError("scale must be positive")
    d = AttnDesc(batch, queries, keys, heads_q, heads_kv, dim, dtype, q_block, max_blocks,
                 sink_blocks, local_blocks, int(bool(backward)), 0.0 if scale is None else scale)
    h = C.c_void_p()
    _check(_lib.spmm_plan_attn(C.byref(d), device, C.byref(h)), "spmm_plan_attn")
    return Plan(h, _attn_expect(d, device))


def _attn_expect(d: AttnDesc, device: int) -> dict:
    """Shapes and types of an attention plan's tensors."""
    import torch
    b, nq, nk, hq, hk, dim = d.batch, d.queries, d.keys, d.heads_q, d.heads_kv, d.dim
    t = torch.bfloat16 if d.dtype == BF16 else torch.float16
    nkb, nqb = -(-nk // 64), -(-nq // d.q_block)
    return {"device": int(device), "attn": {
        "q": ((b, nq, hq, dim), t), "k": ((b, nk, hk, dim), t), "page": ((64, hk, dim), t),
        "lse": ((b, hq, nq), torch.float32), "lists": ((b, hk, nqb, d.max_blocks), torch.int32),
        "table": ((b, nkb), torch.int32), "seq": ((b,), torch.int32), "tree": ((b, nq), torch.int64),
        "slots": b * nkb, "int8": torch.int8, "page8": ((64, hk, dim), torch.int8), "k8": ((b, nk, hk, dim), torch.int8),
        "new": ((b, nq, hk, dim), t)}}


_raw_stream = None
_bind = None

# Marshalling of the attention calls: each tensor is checked against the plan
# (in csrc/binding.cpp: the smallest calls take as long as their marshalling),
# then goes as a pointer, a tensor of heads with strides.


class _PythonChecks:
    """What csrc/binding.cpp does, where that module is not built (a library
    given in SPMM_LIBRARY) or was built for another Python or torch: 0.3 us a
    tensor more."""

    @staticmethod
    def heads(t, want, device, pack=struct.Struct("=4q").pack):
        if t.dtype is not want[1] or t.shape != want[0] or t.get_device() != device:
            return None
        sb, st, sh, sd = t.stride()
        return pack(t.data_ptr(), sb, st, sh) if sd == 1 or not t.numel() else False

    @staticmethod
    def flat(t, want, device):
        if t.dtype is not want[1] or t.shape != want[0] or t.get_device() != device:
            return None
        return t.data_ptr() if t.is_contiguous() else False


def _load_binding():
    global _bind
    import torch
    try:
        from . import _binding
        _bind = _binding if torch.__version__.split("+")[0] == _binding.torch_version else _PythonChecks
    except ImportError:
        _bind = _PythonChecks
    return _bind


def _attn_want(plan: Plan) -> dict:
    want = plan.expect.get("attn")
    if want is None:
        raise ValueError("not a plan of spmm_plan_attn")
    return want


def _refuse(name: str, t, shape, dtype, device):
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}; the plan takes {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the plan takes {shape}")
    raise ValueError(f"{name} must be on cuda:{device}")


def _heads(name: str, t, want, device):
    """A tensor of heads: its strides go along."""
    r = (_bind or _load_binding()).heads(t, want, device)
    if r:
        return r
    if r is None:
        _refuse(name, t, *want, device)
    raise ValueError(f"{name}: the elements of a head must be consecutive")


def _flat(name: str, t, want, device):
    """A contiguous tensor."""
    r = (_bind or _load_binding()).flat(t, want, device)
    if r is None:
        _refuse(name, t, *want, device)
    if r is False:
        raise ValueError(f"{name} must be contiguous")
    return r


def _opt(name: str, t, want, device):
    return None if t is None else _flat(name, t, want, device)


def _stream_of(stream, device):
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    global _raw_stream
    if _raw_stream is None:
        import torch
        # the handle alone where this torch has it: a Stream object takes 2 us
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def spmm_execute_attn_pool(plan: Plan, k, pooled, pooled_scale, lens=None, table=None, first=None,
                           stream=None):
    """Mean keys of the blocks in 8 bits, pooled [slots, heads_kv, dim] int8
    with pooled_scale [slots, heads_kv] float32.  k is [batch, keys, heads_kv,
    dim] (slots = batch * blocks), or with a table [pages, 64, heads_kv, dim]
    (slots = pages).  first [batch]: only the blocks from that key on."""
    w, d = _attn_want(plan), plan.expect["device"]
    pages, slots, kw = 0, w["slots"], w["k"]
    if table is not None:
        pages = slots = k.shape[0]
        kw = ((pages,) + w["page"][0], w["page"][1])
    _, hk, dim = w["page"][0]
    st = _lib.spmm_execute_attn_pool(
        plan.handle, _heads("k", k, kw, d), pages, _flat("pooled", pooled, ((slots, hk, dim), w["int8"]), d),
        _flat("pooled_scale", pooled_scale, ((slots, hk), w["lse"][1]), d), _opt("table", table, w["table"], d),
        _opt("lens", lens, w["seq"], d), _opt("first", first, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_pool")


def spmm_execute_attn_select(plan: Plan, q, pooled, pooled_scale, lists, lens=None, starts=None,
                             table=None, stream=None):
    """lists [batch, heads_kv, query blocks, max_blocks] int32: the blocks of
    the highest scores, ascending, filled up with -1."""
    w, d = _attn_want(plan), plan.expect["device"]
    pages, slots = 0, w["slots"]
    if table is not None:
        pages = slots = pooled.shape[0]
    _, hk, dim = w["page"][0]
    st = _lib.spmm_execute_attn_select(
        plan.handle, _heads("q", q, w["q"], d), _flat("pooled", pooled, ((slots, hk, dim), w["int8"]), d),
        _flat("pooled_scale", pooled_scale, ((slots, hk), w["lse"][1]), d), pages,
        _flat("lists", lists, w["lists"], d), _opt("table", table, w["table"], d), _opt("lens", lens, w["seq"], d),
        _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_select")


def spmm_execute_attn(plan: Plan, q, k, v, lists, o, lse, lens=None, starts=None, stream=None):
    """o (as q) and lse [batch, heads_q, queries] float32 of attention over
    the listed blocks.  Query t stands at position starts + t."""
    w, d = _attn_want(plan), plan.expect["device"]
    qw, kw = w["q"], w["k"]
    st = _lib.spmm_execute_attn(
        plan.handle, _heads("q", q, qw, d), _heads("k", k, kw, d), _heads("v", v, kw, d),
        _flat("lists", lists, w["lists"], d), _heads("o", o, qw, d), _flat("lse", lse, w["lse"], d),
        _opt("lens", lens, w["seq"], d), _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn")


def spmm_execute_attn_backward(plan: Plan, grad, q, k, v, lists, o, lse, dq, dk, dv, lens=None,
                               starts=None, stream=None):
    """dq, dk and dv from grad, the gradient of o; o and lse are the forward
    call's.  The plan must have been made with backward=True."""
    w, d = _attn_want(plan), plan.expect["device"]
    qw, kw = w["q"], w["k"]
    st = _lib.spmm_execute_attn_backward(
        plan.handle, _heads("grad", grad, qw, d), _heads("q", q, qw, d), _heads("k", k, kw, d),
        _heads("v", v, kw, d), _flat("lists", lists, w["lists"], d), _heads("o", o, qw, d),
        _flat("lse", lse, w["lse"], d), _heads("dq", dq, qw, d), _heads("dk", dk, kw, d), _heads("dv", dv, kw, d),
        _opt("lens", lens, w["seq"], d), _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_backward")


def spmm_execute_attn_cache(plan: Plan, q, k, v, o, lse, table=None, lists=None, tree=None, lens=None,
                            starts=None, stream=None):
    """o and lse of new tokens over a cache: k and v are pages [pages, 64,
    heads_kv, dim] with a table [batch, blocks], else [batch, keys, heads_kv,
    dim]; every block, or the lists'.  tree [batch, queries] int64: bit u of a
    drafted token's word is set where it sees drafted token u."""
    w, d = _attn_want(plan), plan.expect["device"]
    pages, qw, kw = 0, w["q"], w["k"]
    if table is not None:
        pages = k.shape[0]
        if pages != v.shape[0]:
            raise ValueError("k and v must have the same pages")
        kw = ((pages,) + w["page"][0], w["page"][1])
    st = _lib.spmm_execute_attn_cache(
        plan.handle, _heads("q", q, qw, d), _heads("k", k, kw, d), _heads("v", v, kw, d), pages,
        _heads("o", o, qw, d), _flat("lse", lse, w["lse"], d), _opt("table", table, w["table"], d),
        _opt("lists", lists, w["lists"], d), _opt("tree", tree, w["tree"], d), _opt("lens", lens, w["seq"], d),
        _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_cache")


def _codes(w, d, k8, v8, k_scale, v_scale, table):
    """Pointers of a cache in 8 bits, and its pages."""
    pages, slots, kw = 0, w["slots"], w["k8"]
    if table is not None:
        pages = slots = k8.shape[0]
        kw = ((pages,) + w["page8"][0], w["page8"][1])
    sw = ((slots, kw[0][2], 64), w["lse"][1])
    return (_heads("k8", k8, kw, d), _heads("v8", v8, kw, d), _flat("k_scale", k_scale, sw, d),
            _flat("v_scale", v_scale, sw, d), pages)


def spmm_execute_attn_write(plan: Plan, k, v, k8, v8, k_scale, v_scale, table=None, lens=None, starts=None,
                            stream=None):
    """New tokens k, v [batch, queries, heads_kv, dim] to a cache in 8 bits, from
    position starts on: k8 and v8 are pages [pages, 64, heads_kv, dim] int8 with a
    table, else [batch, keys, heads_kv, dim]; k_scale and v_scale are [slots,
    heads_kv, 64] float32 (slots = pages, or batch * blocks)."""
    w, d = _attn_want(plan), plan.expect["device"]
    st = _lib.spmm_execute_attn_write(
        plan.handle, _heads("k", k, w["new"], d), _heads("v", v, w["new"], d),
        *_codes(w, d, k8, v8, k_scale, v_scale, table), _opt("table", table, w["table"], d),
        _opt("lens", lens, w["seq"], d), _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_write")


def spmm_execute_attn_read(plan: Plan, k8, v8, k_scale, v_scale, k, v, table=None, lens=None, stream=None):
    """A cache in 8 bits (as spmm_execute_attn_write has it) back to k and v
    [batch, keys, heads_kv, dim]; keys at or past lens are left as they were."""
    w, d = _attn_want(plan), plan.expect["device"]
    st = _lib.spmm_execute_attn_read(
        plan.handle, *_codes(w, d, k8, v8, k_scale, v_scale, table), _heads("k", k, w["k"], d),
        _heads("v", v, w["k"], d), _opt("table", table, w["table"], d), _opt("lens", lens, w["seq"], d),
        _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_read")


def spmm_execute_attn_pool8(plan: Plan, k8, k_scale, pooled, pooled_scale, lens=None, table=None, first=None,
                            stream=None):
    """spmm_execute_attn_pool of the keys of a cache in 8 bits."""
    w, d = _attn_want(plan), plan.expect["device"]
    pages, slots, kw = 0, w["slots"], w["k8"]
    if table is not None:
        pages = slots = k8.shape[0]
        kw = ((pages,) + w["page8"][0], w["page8"][1])
    _, hk, dim = w["page"][0]
    st = _lib.spmm_execute_attn_pool8(
        plan.handle, _heads("k8", k8, kw, d), _flat("k_scale", k_scale, ((slots, hk, 64), w["lse"][1]), d), pages,
        _flat("pooled", pooled, ((slots, hk, dim), w["int8"]), d),
        _flat("pooled_scale", pooled_scale, ((slots, hk), w["lse"][1]), d), _opt("table", table, w["table"], d),
        _opt("lens", lens, w["seq"], d), _opt("first", first, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_pool8")


def spmm_execute_attn_cache8(plan: Plan, q, k8, v8, k_scale, v_scale, o, lse, table=None, lists=None, tree=None,
                             lens=None, starts=None, stream=None):
    """spmm_execute_attn_cache over a cache in 8 bits (as spmm_execute_attn_write
    has it)."""
    w, d = _attn_want(plan), plan.expect["device"]
    qw = w["q"]
    st = _lib.spmm_execute_attn_cache8(
        plan.handle, _heads("q", q, qw, d), *_codes(w, d, k8, v8, k_scale, v_scale, table), _heads("o", o, qw, d),
        _flat("lse", lse, w["lse"], d), _opt("table", table, w["table"], d), _opt("lists", lists, w["lists"], d),
        _opt("tree", tree, w["tree"], d), _opt("lens", lens, w["seq"], d), _opt("starts", starts, w["seq"], d),
        _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_cache8")


def spmm_plan_attn_rope(batch: int, tokens: int, heads_q: int, heads_kv: int, dim: int, freqs, axis=None,
                        dtype: int = BF16, interleaved: bool = False, eps: float = 1e-6, backward: bool = False,
                        axes: int | None = None, device: int = 0) -> Plan:
    """Plan the norm of each head of queries and keys with the rotation of
    len(freqs) pairs of channels: pair p turns by freqs[p] radians a position of
    axis[p] (default: one axis).  Pairs are (p, pairs + p), or neighbours where
    interleaved."""
    f = np.ascontiguousarray(freqs, dtype=np.float64)
    if f.ndim != 1:
        raise ValueError("freqs must be 1-D")
    x = None if axis is None else np.ascontiguousarray(axis, dtype=np.int32)
    if x is not None and x.shape != f.shape:
        raise ValueError("axis must have an entry for each pair")
    if axes is None:
        axes = 1 if x is None or not len(x) else int(x.max()) + 1
    desc = RopeDesc(batch, tokens, heads_q, heads_kv, dim, dtype, len(f), axes, int(bool(interleaved)),
                    int(bool(backward)), eps, _ptr(f), None if x is None else _ptr(x))
    h = C.c_void_p()
    _check(_lib.spmm_plan_attn_rope(C.byref(desc), device, C.byref(h)), "spmm_plan_attn_rope")
    return Plan(h, _rope_expect(desc, device))


def _rope_expect(d: RopeDesc, device: int) -> dict:
    """Shapes and types of a rotation plan's tensors."""
    import torch
    t = torch.bfloat16 if d.dtype == BF16 else torch.float16
    return {"device": int(device), "rope": {
        "q": ((d.batch, d.tokens, d.heads_q, d.dim), t), "k": ((d.batch, d.tokens, d.heads_kv, d.dim), t),
        "weight": ((d.dim,), torch.float32), "positions": ((d.axes, d.batch, d.tokens), torch.int32),
        "seq": ((d.batch,), torch.int32)}}


def _rope_want(plan: Plan) -> dict:
    want = plan.expect.get("rope")
    if want is None:
        raise ValueError("not a plan of spmm_plan_attn_rope")
    return want


def spmm_execute_attn_rope(plan: Plan, q, k, q_out, k_out, q_weight=None, k_weight=None, positions=None, lens=None,
                           starts=None, stream=None):
    """q_out and k_out: q [batch, tokens, heads_q, dim] and k [.., heads_kv, dim]
    normed where there is a weight [dim] float32, and turned.  positions is
    [axes, batch, tokens] int32, by default starts + t.  Tokens whose starts + t
    is not in [0, lens) are left as they were."""
    w, d = _rope_want(plan), plan.expect["device"]
    qw, kw = w["q"], w["k"]
    st = _lib.spmm_execute_attn_rope(
        plan.handle, _heads("q", q, qw, d), _heads("k", k, kw, d), _opt("q_weight", q_weight, w["weight"], d),
        _opt("k_weight", k_weight, w["weight"], d), _heads("q_out", q_out, qw, d), _heads("k_out", k_out, kw, d),
        _opt("positions", positions, w["positions"], d), _opt("lens", lens, w["seq"], d),
        _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_rope")


def spmm_execute_attn_rope_backward(plan: Plan, q_grad, k_grad, q, k, dq, dk, q_weight=None, k_weight=None,
                                    dq_weight=None, dk_weight=None, positions=None, lens=None, starts=None,
                                    stream=None):
    """dq and dk (and dq_weight and dk_weight [dim] float32, where there are
    weights) from the gradients of q_out and k_out; q and k are the forward
    call's inputs (None where there is no weight).  The plan must have been made
    with backward=True."""
    w, d = _rope_want(plan), plan.expect["device"]
    qw, kw, ww = w["q"], w["k"], w["weight"]
    st = _lib.spmm_execute_attn_rope_backward(
        plan.handle, _heads("q_grad", q_grad, qw, d), _heads("k_grad", k_grad, kw, d),
        None if q is None else _heads("q", q, qw, d), None if k is None else _heads("k", k, kw, d),
        _opt("q_weight", q_weight, ww, d), _opt("k_weight", k_weight, ww, d), _heads("dq", dq, qw, d),
        _heads("dk", dk, kw, d), _opt("dq_weight", dq_weight, ww, d), _opt("dk_weight", dk_weight, ww, d),
        _opt("positions", positions, w["positions"], d), _opt("lens", lens, w["seq"], d),
        _opt("starts", starts, w["seq"], d), _stream_of(stream, d))
    if st:
        _check(st, "spmm_execute_attn_rope_backward")
