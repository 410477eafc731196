"""MI355X (gfx950) sparse matrix-vector multiply-accumulate engine, y <- A*x + y.

Thin Python binding over the C ABI of ``include/spmv.h``.  This module only
marshals arguments: every step (validation, statistics, format building, the
SpMV itself) runs in the HIP library ``libspmv_mi355x.so`` built from
``csrc/``.  There is no CPU fallback: if the library cannot be loaded, every
call raises.

    import torch, spmv_storage_formats_amd as spmv
    h = spmv.build("auto", row_ptrs, col_idx, values, num_cols)   # cuda tensors
    h.run(x, y)                  # y += A x on torch's current stream

Weight tables (fp32, fp16 and bf16; token ids int32 or int64):

    q = spmv.build_quant(weights, group_size=128)    # 4 bits per weight, scales per group
    q.run(x, y)                                      # y += W x, one vector or several
    rows = q.lookup(ids)                             # rows of W by token
    rows = spmv.lookup(table, ids, scale=1.0)        # rows of a dense table by token
    dtable = spmv.lookup_grad(drows, ids, num_rows)  # its gradient, by sorted tokens
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import sys
import threading

import numpy as np

__all__ = ["SpmvError", "Handle", "FORMATS", "ARRAYS", "load_library", "analyze", "select",
           "build", "build_coo", "build_tuned", "coo_to_csr", "library_path",
           "declared_functions", "QuantHandle", "build_quant", "build_quant_packed", "lookup",
           "lookup_grad", "lookup_grad_workspace"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_LIB_PATH = os.path.join(_PKG, "libspmv_mi355x.so")
_HEADER = os.path.join(_ROOT, "include", "spmv.h")

FORMATS = {"auto": 0, "coo_atomic": 1, "coo_segmented": 2, "csr_scalar": 3, "csr_vector": 4,
           "ell": 5, "hyb": 6, "jds": 7, "csr_merge": 8, "sell": 9, "ell_xtile": 10,
           "coo_blocked": 11}
FORMAT_NAMES = {v: k for k, v in FORMATS.items()}
# name -> (enum value, numpy dtype)
ARRAYS = {
    "row_ptrs": (0, np.int32), "col_idx": (1, np.int32), "values": (2, np.float32),
    "row_idx": (3, np.int32), "ell_col": (4, np.int32), "ell_val": (5, np.float32),
    "ell_nnz": (6, np.int32), "tail_row": (7, np.int32), "tail_col": (8, np.int32),
    "tail_val": (9, np.float32), "jds_perm": (10, np.int32), "jds_len": (11, np.int32),
    "jds_iter_ptr": (12, np.int32), "jds_col": (13, np.int32), "jds_val": (14, np.float32),
    "len_hist": (15, np.int64), "sell_sect_ptr": (16, np.int32), "sell_col": (17, np.int32),
    "sell_val": (18, np.float32), "xt_run_ptr": (19, np.int32), "xt_runs": (20, np.int32),
    "xt_lidx": (21, np.int16), "bc_chunk_grp": (22, np.int32), "bc_chunk_blk": (23, np.int32),
    "bc_slice_chunk": (24, np.int32), "bc_hot": (25, np.int32), "bc_base": (26, np.int32),
    "bc_pk": (27, np.uint32), "bc_val": (28, np.float32), "bc_wide": (29, np.int32),
    "bc_slice_item": (30, np.int32), "bc_item_chunk": (31, np.int32),
}
CG_NOALLOC_MAX_ROWS = 1048576   # SPMV_CG_NOALLOC_MAX_ROWS in include/spmv.h
BC_BLOCK_ROWS = 32768           # SPMV_BC_BLOCK_ROWS: blocked COO rows per row block
BC_BLOCK_ROWS_TALL = 38912      # SPMV_BC_BLOCK_ROWS_TALL: blocks of balanced layouts
STATUS = {0: "SPMV_OK", 1: "SPMV_ERR_INVALID_ARG", 2: "SPMV_ERR_BAD_ROWPTRS",
          3: "SPMV_ERR_BAD_COLIDX", 4: "SPMV_ERR_BAD_ROWIDX", 5: "SPMV_ERR_TOO_LARGE",
          6: "SPMV_ERR_OOM", 7: "SPMV_ERR_HIP", 8: "SPMV_ERR_DEVICE", 9: "SPMV_ERR_BAD_VALUE"}
DTYPES = {"float32": 0, "float16": 1, "bfloat16": 2, "int32": 3, "int64": 4}   # spmv_dtype


class SpmvError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        self.name = STATUS.get(self.status, f"status {status}")
        msg = _status_string(self.status)
        super().__init__(f"{what}: {self.name} ({msg})" if what else f"{self.name} ({msg})")


class _Opts(ctypes.Structure):
    _fields_ = [("hyb_width", ctypes.c_int32), ("lanes_per_row", ctypes.c_int32),
                ("validate", ctypes.c_int32), ("jds_depth", ctypes.c_int32),
                ("col_blocks", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("max_bytes", ctypes.c_int64)]


class _Stats(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int64), ("num_cols", ctypes.c_int64),
                ("nnz", ctypes.c_int64), ("max_len", ctypes.c_int64),
                ("sum_len_sq", ctypes.c_int64), ("empty_rows", ctypes.c_int64),
                ("col_spread", ctypes.c_int64)]


class _Info(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("hyb_width", ctypes.c_int32),
                ("lanes_per_row", ctypes.c_int32), ("ell_width", ctypes.c_int32),
                ("col_blocks", ctypes.c_int32), ("slice_cols", ctypes.c_int32),
                ("stats", _Stats), ("tail_nnz", ctypes.c_int64), ("num_tiles", ctypes.c_int64),
                ("device_bytes", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("wide_groups", ctypes.c_int64), ("block_rows", ctypes.c_int32),
                ("chunk_entries", ctypes.c_int32), ("hot_slots", ctypes.c_int32),
                ("hot_min_len", ctypes.c_int32), ("work_items", ctypes.c_int32)]


class _TuneEntry(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("col_blocks", ctypes.c_int32),
                ("status", ctypes.c_int32), ("us", ctypes.c_float)]


class _QuantInfo(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int32), ("num_cols", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("zero_points", ctypes.c_int32),
                ("device_bytes", ctypes.c_int64)]


TUNE_MAX = 32


class _TuneReport(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("chosen", ctypes.c_int32),
                ("entry", _TuneEntry * TUNE_MAX)]


_lock = threading.Lock()
_lib = None
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


def library_path() -> str:
    return _LIB_PATH


def declared_functions() -> list[str]:
    """Names of the functions include/spmv.h declares (the library's exports)."""
    with open(_HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(spmv_[a-z_]+)\s*\(", text)))


def load_library():
    """Load the HIP library (building it in-tree first if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            from . import _build
            _build.build()
        lib = ctypes.CDLL(_LIB_PATH)
        P = ctypes.POINTER
        sig = {
            "spmv_opts_default": (None, [P(_Opts)]),
            "spmv_analyze": (ctypes.c_int, [_i32, _i32, _i32, _vp, _vp, _i32, P(_Stats), _vp,
                                            ctypes.c_int64, _vp]),
            "spmv_select": (ctypes.c_int, [P(_Stats), _vp, P(_Opts), P(_i32), P(_i32), P(_i32)]),
            "spmv_build": (ctypes.c_int, [P(_vp), ctypes.c_int, _i32, _i32, _i32, _vp, _vp, _vp,
                                          P(_Opts), _vp]),
            "spmv_build_coo": (ctypes.c_int, [P(_vp), ctypes.c_int, _i32, _i32, _i32, _vp, _vp,
                                              _vp, P(_Opts), _vp]),
            "spmv_coo_to_csr": (ctypes.c_int, [_i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                               _i32, _vp]),
            "spmv_build_tuned": (ctypes.c_int, [P(_vp), _i32, _i32, _i32, _vp, _vp, _vp, P(_Opts),
                                                ctypes.c_uint32, _i32, P(_TuneReport), _vp]),
            "spmv_run": (ctypes.c_int, [_vp, _vp, _vp, _vp]),
            "spmv_cg": (ctypes.c_int, [_vp, _vp, _vp, _i32, ctypes.c_float, P(_i32),
                                       P(ctypes.c_float), _vp]),
            "spmv_cg_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _i32, ctypes.c_float, P(_i32),
                                               P(ctypes.c_float), _vp]),
            "spmv_get_info": (ctypes.c_int, [_vp, P(_Info)]),
            "spmv_array_bytes": (ctypes.c_int, [_vp, ctypes.c_int, P(ctypes.c_size_t)]),
            "spmv_export": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_size_t]),
            "spmv_destroy": (ctypes.c_int, [_vp]),
            "spmv_quant_build": (ctypes.c_int, [P(_vp), _i32, _i32, _i32, _i32, ctypes.c_int,
                                                _vp, _i64, ctypes.c_int, _vp]),
            "spmv_quant_build_packed": (ctypes.c_int, [P(_vp), _i32, _i32, _i32, _vp, _vp,
                                                       ctypes.c_int, _vp, _i32, _vp]),
            "spmv_quant_run_workspace": (ctypes.c_int, [_vp, _i32, ctypes.c_int,
                                                        P(ctypes.c_size_t)]),
            "spmv_quant_run": (ctypes.c_int, [_vp, _i32, _vp, _i64, ctypes.c_int, _vp, _i64,
                                              ctypes.c_int, _i32, _vp, ctypes.c_size_t, _vp]),
            "spmv_quant_lookup": (ctypes.c_int, [_vp, _i64, _vp, ctypes.c_int, ctypes.c_float,
                                                 _vp, _i64, ctypes.c_int, _vp]),
            "spmv_quant_get_info": (ctypes.c_int, [_vp, P(_QuantInfo)]),
            "spmv_quant_array_bytes": (ctypes.c_int, [_vp, ctypes.c_int, P(ctypes.c_size_t)]),
            "spmv_quant_export": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_size_t]),
            "spmv_quant_destroy": (ctypes.c_int, [_vp]),
            "spmv_lookup": (ctypes.c_int, [_i32, _i32, _vp, _i64, ctypes.c_int, _i64, _vp,
                                           ctypes.c_int, ctypes.c_float, _vp, _i64, ctypes.c_int,
                                           _vp]),
            "spmv_lookup_grad_workspace": (ctypes.c_int, [_i32, _i32, _i64,
                                                          P(ctypes.c_size_t)]),
            "spmv_lookup_grad": (ctypes.c_int, [_i32, _i32, _i64, _vp, ctypes.c_int, _vp, _i64,
                                                ctypes.c_int, ctypes.c_float, _i32, _vp, _i64,
                                                ctypes.c_int, _vp, ctypes.c_size_t, _vp]),
            "spmv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "spmv_format_name": (ctypes.c_char_p, [ctypes.c_int]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _status_string(st: int) -> str:
    try:
        return load_library().spmv_status_string(st).decode()
    except Exception:  # pragma: no cover - library not loadable
        return "?"


def _check(st: int, what: str):
    if st != 0:
        raise SpmvError(st, what)


def _opts(hyb_width=0, lanes=0, validate=True, jds_depth=0, max_bytes=0, col_blocks=0) -> _Opts:
    return _Opts(int(hyb_width), int(lanes), 1 if validate else 0, int(jds_depth),
                 int(col_blocks), 0, int(max_bytes))


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}; one of {sorted(FORMATS)}")
        return FORMATS[fmt]
    return int(fmt)


def _dev(t, dtype, name, length=None):
    """Device pointer of a contiguous cuda tensor of `dtype` (0 if empty)."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a cuda tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if length is not None and t.numel() != length:
        raise ValueError(f"{name} has {t.numel()} elements, expected {length}")
    return t.data_ptr() if t.numel() else None


def _stream(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _stats_dict(st: _Stats) -> dict:
    return {k: int(getattr(st, k)) for k, _ in _Stats._fields_}


def analyze(row_ptrs, col_idx, num_cols: int, validate: bool = True, stream=None) -> dict:
    """Input checks + row statistics on the device.  Returns the stats and
    the row-length histogram (numpy int64[max_len + 1])."""
    import torch
    lib = load_library()
    R = row_ptrs.numel() - 1
    rp = _dev(row_ptrs, torch.int32, "row_ptrs")
    ci = _dev(col_idx, torch.int32, "col_idx")
    st = _Stats()
    s = _stream(stream, row_ptrs.device)
    _check(lib.spmv_analyze(R, num_cols, col_idx.numel(), rp, ci, 1 if validate else 0,
                            ctypes.byref(st), None, 0, s), "spmv_analyze")
    hist = np.zeros(st.max_len + 1, np.int64)
    _check(lib.spmv_analyze(R, num_cols, col_idx.numel(), rp, ci, 0, ctypes.byref(st),
                            hist.ctypes.data, hist.size, s), "spmv_analyze")
    out = _stats_dict(st)
    out["hist"] = hist
    return out


def select(stats: dict, hist, hyb_width: int = 0, lanes: int = 0):
    """The library's format selector (host function): (format, K, lanes)."""
    lib = load_library()
    st = _Stats(*(int(stats[k]) for k, _ in _Stats._fields_))
    h = np.ascontiguousarray(hist, np.int64)
    if h.size != st.max_len + 1:
        raise ValueError("hist must have max_len + 1 entries")
    f, K, L = _i32(), _i32(), _i32()
    o = _opts(hyb_width, lanes)
    _check(lib.spmv_select(ctypes.byref(st), h.ctypes.data, ctypes.byref(o), ctypes.byref(f),
                           ctypes.byref(K), ctypes.byref(L)), "spmv_select")
    return FORMAT_NAMES[f.value], K.value, L.value


class Handle:
    """A built matrix.  Owns device copies of its format arrays."""

    def __init__(self, ptr: int, device):
        self._ptr = ctypes.c_void_p(ptr)
        self.device = device
        lib = load_library()
        info = _Info()
        _check(lib.spmv_get_info(self._ptr, ctypes.byref(info)), "spmv_get_info")
        self.info = {"format": FORMAT_NAMES[info.format], "hyb_width": info.hyb_width,
                     "lanes_per_row": info.lanes_per_row, "ell_width": info.ell_width,
                     "col_blocks": info.col_blocks, "slice_cols": info.slice_cols,
                     "tail_nnz": info.tail_nnz, "num_tiles": info.num_tiles,
                     "device_bytes": info.device_bytes, "groups": info.groups,
                     "wide_groups": info.wide_groups, "block_rows": info.block_rows,
                     "chunk_entries": info.chunk_entries, "hot_slots": info.hot_slots,
                     "hot_min_len": info.hot_min_len, "work_items": info.work_items,
                     **_stats_dict(info.stats)}

    @property
    def format(self) -> str:
        return self.info["format"]

    @property
    def num_rows(self) -> int:
        return self.info["num_rows"]

    @property
    def num_cols(self) -> int:
        return self.info["num_cols"]

    @property
    def nnz(self) -> int:
        return self.info["nnz"]

    def run(self, x, y, stream=None):
        """y <- A x + y, enqueued on `stream` (default: torch's current stream)."""
        import torch
        if self._ptr is None:
            raise RuntimeError("handle destroyed")
        xp = _dev(x, torch.float32, "x", self.num_cols)
        yp = _dev(y, torch.float32, "y", self.num_rows)
        if xp is not None and yp is not None:
            xs, xe = xp, xp + 4 * self.num_cols
            ys, ye = yp, yp + 4 * self.num_rows
            if xs < ye and ys < xe:
                raise ValueError("x and y must not overlap")
        _check(load_library().spmv_run(self._ptr, xp, yp, _stream(stream, y.device)),
               "spmv_run")
        return y

    def cg(self, b, x, max_iter: int = 1000, rtol: float = 1e-6, stream=None):
        """Conjugate gradient for A x = b (A square, symmetric positive definite).
        x holds the initial guess and receives the solution.  Returns
        (iterations, ||b - A x|| / ||b|| of the recurrence)."""
        import torch
        bp = _dev(b, torch.float32, "b", self.num_rows)
        xp = _dev(x, torch.float32, "x", self.num_rows)
        it = _i32()
        rr = ctypes.c_float()
        _check(load_library().spmv_cg(self._ptr, bp, xp, int(max_iter), float(rtol),
                                      ctypes.byref(it), ctypes.byref(rr),
                                      _stream(stream, x.device)), "spmv_cg")
        return it.value, rr.value

    def cg_noalloc(self, b, x, max_iter: int = 1000, rtol: float = 1e-6, stream=None):
        """The same solve as cg() on the library's static per-GPU workspace
        (spmv_cg_noalloc: no device allocation, at most CG_NOALLOC_MAX_ROWS rows;
        calls overlapping on one GPU race)."""
        import torch
        bp = _dev(b, torch.float32, "b", self.num_rows)
        xp = _dev(x, torch.float32, "x", self.num_rows)
        it = _i32()
        rr = ctypes.c_float()
        _check(load_library().spmv_cg_noalloc(self._ptr, bp, xp, int(max_iter), float(rtol),
                                              ctypes.byref(it), ctypes.byref(rr),
                                              _stream(stream, x.device)), "spmv_cg_noalloc")
        return it.value, rr.value

    def array(self, name: str) -> np.ndarray:
        """Copy one of the handle's arrays to a numpy array (bit-exact)."""
        which, dtype = ARRAYS[name]
        lib = load_library()
        n = ctypes.c_size_t()
        _check(lib.spmv_array_bytes(self._ptr, which, ctypes.byref(n)), "spmv_array_bytes")
        out = np.empty(n.value // np.dtype(dtype).itemsize, dtype)
        _check(lib.spmv_export(self._ptr, which, out.ctypes.data if out.size else None,
                               n.value), "spmv_export")
        return out

    def has_array(self, name: str) -> bool:
        n = ctypes.c_size_t()
        _check(load_library().spmv_array_bytes(self._ptr, ARRAYS[name][0], ctypes.byref(n)),
               "spmv_array_bytes")
        return n.value > 0 or name == "len_hist"

    def close(self):
        if sys.is_finalizing():
            return  # the HIP runtime may already be gone; the process frees it
        if getattr(self, "_ptr", None) is not None and _lib is not None:
            _lib.spmv_destroy(self._ptr)
        self._ptr = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def build(fmt, row_ptrs, col_idx, values, num_cols: int, *, hyb_width: int = 0, lanes: int = 0,
          validate: bool = True, jds_depth: int = 0, max_bytes: int = 0, col_blocks: int = 0,
          stream=None) -> Handle:
    """Build a handle in `fmt` ("auto" = selector) from CSR cuda tensors."""
    import torch
    lib = load_library()
    R = row_ptrs.numel() - 1
    nnz = col_idx.numel()
    rp = _dev(row_ptrs, torch.int32, "row_ptrs")
    ci = _dev(col_idx, torch.int32, "col_idx")
    va = _dev(values, torch.float32, "values", nnz)
    out = ctypes.c_void_p()
    o = _opts(hyb_width, lanes, validate, jds_depth, max_bytes, col_blocks)
    _check(lib.spmv_build(ctypes.byref(out), _fmt(fmt), R, int(num_cols), nnz, rp, ci, va,
                          ctypes.byref(o), _stream(stream, row_ptrs.device)), "spmv_build")
    return Handle(out.value, row_ptrs.device)


def build_coo(fmt, row_idx, col_idx, values, num_rows: int, num_cols: int, *, hyb_width: int = 0,
              lanes: int = 0, validate: bool = True, jds_depth: int = 0, max_bytes: int = 0,
              col_blocks: int = 0, stream=None) -> Handle:
    """Build a handle from COO cuda tensors (converted to CSR on the device)."""
    import torch
    lib = load_library()
    nnz = col_idx.numel()
    ri = _dev(row_idx, torch.int32, "row_idx", nnz)
    ci = _dev(col_idx, torch.int32, "col_idx")
    va = _dev(values, torch.float32, "values", nnz)
    out = ctypes.c_void_p()
    o = _opts(hyb_width, lanes, validate, jds_depth, max_bytes, col_blocks)
    _check(lib.spmv_build_coo(ctypes.byref(out), _fmt(fmt), int(num_rows), int(num_cols), nnz,
                              ri, ci, va, ctypes.byref(o), _stream(stream, col_idx.device)),
           "spmv_build_coo")
    return Handle(out.value, col_idx.device)


def coo_to_csr(row_idx, col_idx, values, num_rows: int, num_cols: int, validate: bool = True,
               stream=None):
    """COO -> CSR on the device.  Returns (row_ptrs, col_idx, values) tensors."""
    import torch
    lib = load_library()
    nnz = col_idx.numel()
    dev = col_idx.device
    rp = torch.empty(num_rows + 1, dtype=torch.int32, device=dev)
    co = torch.empty(nnz, dtype=torch.int32, device=dev)
    vo = torch.empty(nnz, dtype=torch.float32, device=dev)
    _check(lib.spmv_coo_to_csr(int(num_rows), int(num_cols), nnz,
                               _dev(row_idx, torch.int32, "row_idx", nnz),
                               _dev(col_idx, torch.int32, "col_idx"),
                               _dev(values, torch.float32, "values", nnz),
                               rp.data_ptr(), _dev(co, torch.int32, "out"),
                               _dev(vo, torch.float32, "out"), 1 if validate else 0,
                               _stream(stream, dev)), "spmv_coo_to_csr")
    return rp, co, vo


def build_tuned(row_ptrs, col_idx, values, num_cols: int, *, formats=None, runs: int = 5,
                hyb_width: int = 0, lanes: int = 0, validate: bool = True, jds_depth: int = 0,
                stream=None):
    """Empirical selector: time every candidate format on this matrix, keep the
    fastest.  Returns (handle, report) where report is a list of dicts
    {format, col_blocks, status, us} and report[i]["chosen"] marks the winner."""
    import torch
    lib = load_library()
    R = row_ptrs.numel() - 1
    nnz = col_idx.numel()
    mask = 0
    for f in (formats or []):
        mask |= 1 << _fmt(f)
    out = ctypes.c_void_p()
    rep = _TuneReport()
    o = _opts(hyb_width, lanes, validate, jds_depth, 0, 0)
    _check(lib.spmv_build_tuned(ctypes.byref(out), R, int(num_cols), nnz,
                                _dev(row_ptrs, torch.int32, "row_ptrs"),
                                _dev(col_idx, torch.int32, "col_idx"),
                                _dev(values, torch.float32, "values", nnz), ctypes.byref(o),
                                mask, int(runs), ctypes.byref(rep),
                                _stream(stream, row_ptrs.device)), "spmv_build_tuned")
    report = []
    for i in range(rep.count):
        e = rep.entry[i]
        report.append({"format": FORMAT_NAMES[e.format], "col_blocks": e.col_blocks,
                       "status": STATUS.get(e.status, e.status), "us": float(e.us),
                       "chosen": i == rep.chosen})
    return Handle(out.value, row_ptrs.device), report


# ------------------------------------------------------------- weight tables

_FLOATS = ("float32", "float16", "bfloat16")
_IDS = ("int32", "int64")
_codes = {}     # (torch dtype, names allowed) -> spmv_dtype, filled by _kind


def _kind(dtype, allowed, name):
    """spmv_dtype of a torch dtype, which must be one of `allowed`."""
    hit = _codes.get((dtype, allowed))
    if hit is None:
        s = str(dtype).replace("torch.", "")
        if s not in allowed:
            raise TypeError(f"{name} must be one of {', '.join(allowed)}, got {dtype}")
        hit = _codes[(dtype, allowed)] = DTYPES[s]
    return hit


def _fits(what, *sizes):
    """Refuse sizes that the ABI's int32 arguments would wrap."""
    for n in sizes:
        if n > 0x7fffffff:
            raise SpmvError(5, what)
        if n < -0x80000000:
            raise SpmvError(1, what)


def _rows(t, name, index, rows, cols):
    """A cuda matrix [rows, cols] whose rows are contiguous (rows None: any number), on
    device `index` (None: any): (pointer, row stride, spmv_dtype, end of its memory)."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a cuda tensor")
    kind = _kind(t.dtype, _FLOATS, name)
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                         f"({'any' if rows is None else rows}, {cols})")
    n = shape[0]
    ld, step = t.stride()
    if (step != 1 and cols > 1) or (ld < cols and n > 1):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    if n == 0 or cols == 0:
        return None, ld, kind, 0
    p = t.data_ptr()
    return p, ld, kind, p + ((n - 1) * ld + cols) * (2 if kind else 4)


def _token_ids(ids, index=None):
    """(pointer, count, spmv_dtype, end) of contiguous token ids of any shape."""
    import torch
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise TypeError("ids must be a cuda tensor")
    kind = _kind(ids.dtype, _IDS, "ids")
    if index is not None and ids.get_device() != index:
        raise ValueError(f"ids are on {ids.device}, expected cuda:{index}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    n = ids.numel()
    if n == 0:
        return None, 0, kind, 0
    p = ids.data_ptr()
    return p, n, kind, p + n * (8 if kind == 4 else 4)


def _apart(a, b, what):
    """Refuse tensors whose memory overlaps.  Column ranges of one buffer that lie side
    by side (equal row strides) do not."""
    a0, b0 = a.data_ptr(), b.data_ptr()
    a1, b1 = a0 + _span(a), b0 + _span(b)
    if a0 >= b1 or b0 >= a1 or a0 == a1 or b0 == b1:
        return
    if a.dim() == 2 and b.dim() == 2:
        step = a.stride(0) * a.element_size()
        if step == b.stride(0) * b.element_size() and step > 0:
            at = (b0 - a0) % step
            if at >= a.shape[1] * a.element_size() and at + b.shape[1] * b.element_size() <= step:
                return
    raise ValueError(f"{what} must not overlap")


def _span(t):
    """Bytes from a tensor's first element to behind its last."""
    if t.numel() == 0:
        return 0
    return t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _stream_of(index, stream, *made):
    """Stream handle for work on device `index` (the current device).  Tensors in `made`
    were allocated for the call on torch's current stream: where the work runs on another
    one, it waits for that stream, and their memory is not reused before it is done."""
    import torch
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # makes no Stream object
        return raw(index) if raw else torch.cuda.current_stream(index).cuda_stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    current = torch.cuda.current_stream(index)
    if made and handle != current.cuda_stream:
        other = (stream if isinstance(stream, torch.cuda.Stream)
                 else torch.cuda.ExternalStream(handle, device=index))
        other.wait_stream(current)      # an allocation may still be in use there
        for t in made:
            t.record_stream(other)
    return handle


def _workspace(t, need, index):
    """(pointer, bytes) of a contiguous uint8 cuda tensor of at least `need` bytes."""
    import torch
    p = _dev(t, torch.uint8, "workspace")
    size = t.numel()
    if size < need or t.get_device() != index or (p or 0) % 16:
        raise ValueError(f"workspace must hold {need} bytes on cuda:{index}, 16-byte aligned")
    return p, size


def _elsewhere(index):
    """Whether another device than `index` is current."""
    import torch
    return torch.cuda.current_device() != index


class QuantHandle:
    """A matrix in 4 bits per weight: W[r, c] = scale[r, g] * (code[r, c] - zero[r, g])
    with g = c // group_size.  Owns its device arrays."""

    ARRAYS = {"codes": 0, "scales": 1, "zero_points": 2}

    def __init__(self, ptr: int, device, scale_dtype):
        self._ptr = ctypes.c_void_p(ptr)
        self.device = device
        self.scale_dtype = scale_dtype
        info = _QuantInfo()
        _check(load_library().spmv_quant_get_info(self._ptr, ctypes.byref(info)),
               "spmv_quant_get_info")
        self.info = {k: int(getattr(info, k)) for k, _ in _QuantInfo._fields_
                     if k != "scale_dtype"}
        self.num_rows = info.num_rows
        self.num_cols = info.num_cols
        self.group_size = info.group_size
        self._need = {}     # (vectors, spmv_dtype) -> bytes of workspace

    def _live(self):
        if self._ptr is None:
            raise RuntimeError("handle destroyed")
        return self._ptr

    def run_workspace(self, n: int, dtype) -> int:
        """Bytes of workspace that run needs for n vectors of `dtype` (0 for few)."""
        kind = _kind(dtype, _FLOATS, "dtype")
        hit = self._need.get((n, kind))
        if hit is None:
            _fits("spmv_quant_run_workspace", n)
            size = ctypes.c_size_t()
            _check(load_library().spmv_quant_run_workspace(self._live(), n, kind,
                                                           ctypes.byref(size)),
                   "spmv_quant_run_workspace")
            hit = self._need[(n, kind)] = size.value
        return hit

    def run(self, x, y, *, accumulate: bool = True, workspace=None, stream=None):
        """y <- W x + y (accumulate) or y <- W x, enqueued on `stream` (default: torch's
        current stream).  x [C] and y [R], or x [n, C] and y [n, R] for n vectors; y of
        x's type or fp32.  `workspace`: a contiguous uint8 cuda tensor of at least
        run_workspace() bytes, for this call alone until its work is done (default:
        allocated for the call where it needs one)."""
        ptr = self._live()
        try:
            one = x.dim() == 1 and y.dim() == 1
        except AttributeError:
            raise TypeError("x and y must be cuda tensors") from None
        if one:
            self.run(x[None], y[None], accumulate=accumulate, workspace=workspace,
                     stream=stream)
            return y
        index = self.device.index
        if _elsewhere(index):
            import torch
            with torch.cuda.device(index):
                return self.run(x, y, accumulate=accumulate, workspace=workspace,
                                stream=stream)
        xp, x_ld, xk, xe = _rows(x, "x", index, None, self.num_cols)
        n = x.shape[0]
        yp, y_ld, yk, ye = _rows(y, "y", index, n, self.num_rows)
        if yk != xk and yk != 0:
            raise TypeError(f"y must be {x.dtype} or torch.float32, got {y.dtype}")
        if xe and ye and xp < ye and yp < xe:
            _apart(x, y, "x and y")
        need = self.run_workspace(n, x.dtype)
        wp, size, made = None, 0, ()
        if need:
            if workspace is None:
                import torch
                workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
                made = (workspace,)
                wp, size = workspace.data_ptr(), need
            else:
                wp, size = _workspace(workspace, need, index)
                _apart(workspace, x, "workspace and x")
                _apart(workspace, y, "workspace and y")
        _check(load_library().spmv_quant_run(ptr, n, xp, x_ld, xk, yp, y_ld, yk,
                                             1 if accumulate else 0, wp, size,
                                             _stream_of(index, stream, *made)),
               "spmv_quant_run")
        return y

    def lookup(self, ids, out=None, *, scale: float = 1.0, dtype=None, stream=None):
        """Rows of the matrix by token: out[t, :] = scale * W[ids[t], :], zeros for ids
        outside [0, R).  Returns `out` (default: a new tensor ids.shape + [C] of `dtype`,
        fp32 unless given)."""
        import torch
        ptr = self._live()
        index = self.device.index
        if _elsewhere(index):
            with torch.cuda.device(index):
                return self.lookup(ids, out, scale=scale, dtype=dtype, stream=stream)
        ip, n, ik, ie = _token_ids(ids, index)
        made = ()
        if out is None:
            out = torch.empty((*ids.shape, self.num_cols), dtype=dtype or torch.float32,
                              device=self.device)
            made = (out,)
        flat = _by_token(out, ids, self.num_cols, "out", dtype)
        op, ld, ok, oe = _rows(flat, "out", index, n, self.num_cols)
        if ie and oe and ip < oe and op < ie:
            _apart(ids, flat, "ids and out")
        _check(load_library().spmv_quant_lookup(ptr, n, ip, ik, scale, op, ld, ok,
                                                _stream_of(index, stream, *made)),
               "spmv_quant_lookup")
        return out

    def array(self, name: str) -> np.ndarray:
        """Copy one of the matrix's arrays to a numpy array: "codes" (uint8 [R, ceil(C/2)],
        the even column in the low half), "scales" (float32 values [R, groups]) or
        "zero_points" (uint8 [R, groups]; empty without zero points)."""
        import torch
        ptr = self._live()
        lib = load_library()
        which = self.ARRAYS[name]
        n = ctypes.c_size_t()
        _check(lib.spmv_quant_array_bytes(ptr, which, ctypes.byref(n)), "spmv_quant_array_bytes")
        raw = np.empty(n.value, np.uint8)
        with torch.cuda.device(self.device):
            _check(lib.spmv_quant_export(ptr, which, raw.ctypes.data if raw.size else None,
                                         n.value), "spmv_quant_export")
        if name == "scales":
            if raw.size == 0:
                return np.empty((self.num_rows, self.info["num_groups"]), np.float32)
            raw = torch.from_numpy(raw).view(self.scale_dtype).float().numpy()
        if name == "codes":
            return raw.reshape(self.num_rows, (self.num_cols + 1) // 2)
        return raw.reshape(self.num_rows, -1) if raw.size else raw

    def close(self):
        if sys.is_finalizing():
            return  # the HIP runtime may already be gone; the process frees it
        if getattr(self, "_ptr", None) is not None and _lib is not None:
            _lib.spmv_quant_destroy(self._ptr)
        self._ptr = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _by_token(t, ids, cols, name, dtype=None):
    """A tensor of shape ids.shape + [cols] as a matrix over the tokens."""
    import torch
    if not isinstance(t, torch.Tensor) or t.shape != (*ids.shape, cols):
        raise ValueError(f"{name} must be a tensor of shape {(*ids.shape, cols)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, dtype says {dtype}")
    if t.dim() == 2:
        return t
    try:
        return t.view(ids.numel(), cols)
    except RuntimeError:
        raise ValueError(f"{name}'s rows must lie at one stride") from None


def build_quant(weights, *, group_size: int = 128, zero_points: bool = False, scale_dtype=None,
                stream=None) -> QuantHandle:
    """Quantise a dense cuda matrix [R, C] (fp32, fp16 or bf16) to 4 bits per weight with a
    scale, and with `zero_points` a zero point, per row and group of `group_size` columns
    (32, 64 or a multiple of 128).  Scales are kept in `scale_dtype` (default: weights')."""
    import torch
    if not isinstance(weights, torch.Tensor) or weights.dim() != 2:
        raise ValueError("weights must be a matrix")
    R, C = weights.shape
    _fits("spmv_quant_build", R, C, int(group_size))
    wp, ld, wk, _ = _rows(weights, "weights", None, R, C)
    scale_dtype = scale_dtype or weights.dtype
    sk = _kind(scale_dtype, _FLOATS, "scale_dtype")
    out = ctypes.c_void_p()
    with torch.cuda.device(weights.device):
        _check(load_library().spmv_quant_build(
            ctypes.byref(out), R, C, int(group_size), 1 if zero_points else 0, sk, wp, ld, wk,
            _stream_of(weights.get_device(), stream)), "spmv_quant_build")
    return QuantHandle(out.value, weights.device, scale_dtype)


def build_quant_packed(codes, scales, num_cols: int, *, group_size: int = 128, zero_points=None,
                       validate: bool = True, stream=None) -> QuantHandle:
    """The handle of a matrix that is quantised already: codes uint8 [R, ceil(num_cols/2)]
    (the even column in the low half of a byte), scales [R, ceil(num_cols/group_size)]
    (fp32, fp16 or bf16) and zero_points uint8 like scales (None: 8 everywhere)."""
    import torch
    num_cols, group_size = int(num_cols), int(group_size)
    _fits("spmv_quant_build_packed", num_cols, group_size)
    cp = _dev(codes, torch.uint8, "codes")
    if codes.dim() != 2 or num_cols < 0 or codes.shape[1] != (num_cols + 1) // 2:
        raise ValueError(f"codes must be [R, {(num_cols + 1) // 2}], got {tuple(codes.shape)}")
    R = codes.shape[0]
    _fits("spmv_quant_build_packed", R)
    if group_size <= 0:
        raise ValueError("group_size must be positive")
    shape = (R, -(-num_cols // group_size))
    sk = _kind(getattr(scales, "dtype", None), _FLOATS, "scales")
    sp = _dev(scales, scales.dtype, "scales")
    zp = None if zero_points is None else _dev(zero_points, torch.uint8, "zero_points")
    for t, name in ((scales, "scales"), (zero_points, "zero_points")):
        if t is not None and (tuple(t.shape) != shape or t.device != codes.device):
            raise ValueError(f"{name} must be {shape} on {codes.device}, got "
                             f"{tuple(t.shape)} on {t.device}")
    out = ctypes.c_void_p()
    with torch.cuda.device(codes.device):
        _check(load_library().spmv_quant_build_packed(
            ctypes.byref(out), R, num_cols, group_size, cp, sp, sk, zp, 1 if validate else 0,
            _stream_of(codes.get_device(), stream)), "spmv_quant_build_packed")
    return QuantHandle(out.value, codes.device, scales.dtype)


def lookup(table, ids, out=None, *, scale: float = 1.0, dtype=None, stream=None):
    """Rows of a dense table [V, D] by token: out[t, :] = scale * table[ids[t], :], zeros for
    ids outside [0, V) (padded positions).  Returns `out` (default: a new tensor
    ids.shape + [D] of `dtype`, the table's unless given).  Records no autograd graph:
    lookup_grad is its backward pass."""
    import torch
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a matrix")
    V, D = table.shape
    _fits("spmv_lookup", V, D)
    tp, t_ld, tk, te = _rows(table, "table", None, V, D)
    index = table.get_device()
    if _elsewhere(index):
        with torch.cuda.device(index):
            return lookup(table, ids, out, scale=scale, dtype=dtype, stream=stream)
    ip, n, ik, ie = _token_ids(ids, index)
    made = ()
    if out is None:
        out = torch.empty((*ids.shape, D), dtype=dtype or table.dtype, device=table.device)
        made = (out,)
    flat = _by_token(out, ids, D, "out", dtype)
    op, o_ld, ok, oe = _rows(flat, "out", index, n, D)
    if not made:
        if te and oe and tp < oe and op < te:
            _apart(table, flat, "table and out")
        if ie and oe and ip < oe and op < ie:
            _apart(ids, flat, "ids and out")
    _check(load_library().spmv_lookup(V, D, tp, t_ld, tk, n, ip, ik, scale, op, o_ld, ok,
                                      _stream_of(index, stream, *made)), "spmv_lookup")
    return out


def lookup_grad_workspace(num_tokens: int, num_rows: int, num_cols: int) -> int:
    """Bytes of workspace that lookup_grad needs for these sizes."""
    return _workspace_bytes(int(num_tokens), int(num_rows), int(num_cols))


@functools.lru_cache(maxsize=64)
def _workspace_bytes(n, rows, cols):
    _fits("spmv_lookup_grad_workspace", rows, cols, n)    # n: 64 bits there, 31 allowed
    size = ctypes.c_size_t()
    _check(load_library().spmv_lookup_grad_workspace(rows, cols, n, ctypes.byref(size)),
           "spmv_lookup_grad_workspace")
    return size.value


def lookup_grad(grad, ids, num_rows: int, out=None, *, scale: float = 1.0,
                accumulate: bool = False, dtype=None, workspace=None, stream=None):
    """Gradient of lookup with respect to its table: out[v, :] = scale * the sum of grad[t, :]
    over the tokens t with ids[t] = v, added to `out` with `accumulate`.  grad is ids.shape +
    [D]; ids outside [0, num_rows) contribute nothing.  Returns `out` (default: a new tensor
    [num_rows, D] of `dtype`, grad's unless given).  `workspace`: a contiguous uint8 cuda
    tensor of at least lookup_grad_workspace() bytes, for this call alone until its work is
    done (default: allocated for the call)."""
    import torch
    num_rows = int(num_rows)
    if not isinstance(grad, torch.Tensor) or not grad.is_cuda or grad.dim() < 1:
        raise TypeError("grad must be a cuda tensor")
    index, D = grad.get_device(), grad.shape[-1]
    if _elsewhere(index):
        with torch.cuda.device(index):
            return lookup_grad(grad, ids, num_rows, out, scale=scale, accumulate=accumulate,
                               dtype=dtype, workspace=workspace, stream=stream)
    ip, n, ik, ie = _token_ids(ids, index)
    gp, g_ld, gk, ge = _rows(_by_token(grad, ids, D, "grad"), "grad", index, n, D)
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")
    _fits("spmv_lookup_grad", num_rows, D)
    made = []
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty(num_rows, D, dtype=dtype or grad.dtype, device=grad.device)
        made.append(out)
    elif dtype is not None and isinstance(out, torch.Tensor) and out.dtype != dtype:
        raise TypeError(f"out is {out.dtype}, dtype says {dtype}")
    op, o_ld, ok, oe = _rows(out, "out", index, num_rows, D)
    if not made:
        _apart(grad, out, "grad and out")
        _apart(ids, out, "ids and out")
    need = _workspace_bytes(n, num_rows, D)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=grad.device)
        made.append(workspace)
        wp, size = workspace.data_ptr(), need
    else:
        wp, size = _workspace(workspace, need, index)
        for t, name in ((out, "out"), (grad, "grad"), (ids, "ids")):
            _apart(workspace, t, f"workspace and {name}")
    _check(load_library().spmv_lookup_grad(
        num_rows, D, n, ip, ik, gp, g_ld, gk, scale, 1 if accumulate else 0, op, o_ld, ok, wp,
        size, _stream_of(index, stream, *made)), "spmv_lookup_grad")
    return out
