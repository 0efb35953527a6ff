"""Thin Python binding of libfathom (include/fathom.h).

Argument marshalling only: every function takes torch tensors, checks dtype,
device and contiguity, passes raw pointers and the current CUDA stream to the
C ABI of the same name, and raises ``FathomError`` on a non-zero status.  All
computation runs in the CUDA kernels of libfathom; there is no fallback: if
the library is missing or CUDA is unavailable the call fails.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# FATHOM_LIB names another build of the same library (e.g. the debug build with
# bounds checks, libfathom_debug.so) to load instead of the default one.
LIB_PATH = os.environ.get("FATHOM_LIB") or os.path.join(_PKG, "_build", "libfathom.so")

F32, BF16, F16 = 0, 1, 2
WS_SCAN_TOPK, WS_SPARSE_ATTN, WS_DENSE_ATTN, WS_KLT_ONLINE = 0, 1, 2, 3
SRC_STORE, SRC_STAGING = 0, 1
MAX_D, MAX_G, MAX_K = 128, 8, 2048

# (name, restype, argtypes) of every symbol include/fathom.h declares
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class Shape(ctypes.Structure):
    _fields_ = [("units", ctypes.c_int32), ("n", ctypes.c_int32), ("D", ctypes.c_int32),
                ("G", ctypes.c_int32), ("k", ctypes.c_int32), ("n_sink", ctypes.c_int32),
                ("n_recent", ctypes.c_int32), ("n_cap", ctypes.c_int32), ("scan_ctas_per_sm", ctypes.c_int32)]

    def __repr__(self):
        return (f"Shape(units={self.units}, n={self.n}, D={self.D}, G={self.G}, k={self.k}, "
                f"n_sink={self.n_sink}, n_recent={self.n_recent}, n_cap={self.n_cap}, "
                f"scan_ctas_per_sm={self.scan_ctas_per_sm})")

    @property
    def cap(self) -> int:
        """Tokens the per-unit arrays are laid out for."""
        return self.n_cap if self.n_cap > 0 else self.n


class Prompts(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("seqs", "heads", "kv_heads", "D", "dtype", "total_q", "total_k")] + \
               [(f, ctypes.c_int64) for f in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head",
                                              "out_token", "out_head")]


class Pages(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("seqs", "kv_heads", "D", "dtype", "page_tokens", "num_pages",
                                              "max_pages")] + \
               [(f, ctypes.c_int64) for f in ("page_stride", "head_stride", "token_stride")]

    def __repr__(self):
        return type(self).__name__ + "(" + ", ".join(f"{f}={getattr(self, f)}" for f, _ in self._fields_) + ")"

    @property
    def units(self) -> int:
        return self.seqs * self.kv_heads

    @property
    def cap(self) -> int:
        """Tokens a row of the page table can name."""
        return self.max_pages * self.page_tokens


class NibblePages(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("seqs", "kv_heads", "D", "page_tokens", "num_pages", "max_pages")] + \
               [(f, ctypes.c_int64) for f in ("page_stride", "head_stride")]

    __repr__ = Pages.__repr__
    units = Pages.units
    cap = Pages.cap


class Rope(ctypes.Structure):
    _fields_ = [("table", _vp), ("rows", _i32), ("rot", _i32), ("interleaved", _i32), ("positions", _vp), ("q", _vp),
                ("q_out", _vp), ("q_heads", _i32), ("q_dtype", _i32), ("q_token", _i64), ("q_head", _i64),
                ("out_token", _i64), ("out_head", _i64)]


RUN_FIELDS = ("src_word", "n_words", "dst_word", "src_scale", "n_scales", "dst_scale")
RUN_BYTES = 24

SIGNATURES = {
    "fathom_calibrate": (ctypes.c_int, [_i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "fathom_calibrate_klt": (ctypes.c_int, [_i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "fathom_rotate_keys": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, ctypes.c_int, _i32, _vp, _vp, _vp, _vp]),
    "fathom_rotate_query": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _i32, _vp, _vp, _vp]),
    "fathom_quantize_pack": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, ctypes.c_int, _vp, _vp, _vp]),
    "fathom_append_block": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, ctypes.c_int, _i32, _i32, _vp, _vp, _vp]),
    "fathom_plan": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fathom_plan_fixed": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "fathom_gather": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _sz, _sz, _vp]),
    "fathom_scan_topk": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, ctypes.c_int, _sz, _sz, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fathom_scan": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, ctypes.c_int, _sz, _sz, _vp, _vp, _vp, _vp,
                                   _sz, _vp]),
    "fathom_select": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, ctypes.c_int, _sz, _sz, _vp, _vp, _vp, _vp,
                                     _vp, _sz, _vp]),
    "fathom_exact_topk": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fathom_sparse_attn": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fathom_dense_attn": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fathom_sparse_attn_planes": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                                 _vp]),
    "fathom_sparse_attn_noalloc": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp]),
    "fathom_klt_online": (ctypes.c_int, [ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fathom_prefill_attn": (ctypes.c_int, [ctypes.POINTER(Prompts), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fathom_paged_append": (ctypes.c_int, [ctypes.POINTER(Pages), _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _vp, _vp,
                                           _vp]),
    "fathom_paged_attn": (ctypes.c_int, [ctypes.POINTER(Pages), _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz,
                                         _vp]),
    "fathom_paged_evict": (ctypes.c_int, [ctypes.POINTER(Pages), _vp, _vp, _vp, _vp, _vp, _sz, _i32, _i32, _i32, _vp,
                                          _i32, _vp, _vp, _vp, _sz, _vp]),
    "fathom_paged_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Pages), _i32, ctypes.c_int]),
    "fathom_paged_append_rope": (ctypes.c_int, [ctypes.POINTER(Pages), _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _vp,
                                                _vp, ctypes.POINTER(Rope), _vp]),
    "fathom_nibble_append": (ctypes.c_int, [ctypes.POINTER(NibblePages), _vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _vp,
                                            _vp, ctypes.POINTER(Rope), _vp]),
    "fathom_nibble_read": (ctypes.c_int, [ctypes.POINTER(NibblePages), _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i64,
                                          _i64, _vp]),
    "fathom_nibble_attn": (ctypes.c_int, [ctypes.POINTER(NibblePages), _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fathom_nibble_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(NibblePages), _i32]),
    "fathom_wait_status": (ctypes.c_int, []),
    "fathom_rel_err": (ctypes.c_int, [_i32, _i32, _vp, _vp, _vp, _vp]),
    "fathom_set_overlap": (ctypes.c_int, [_i32, _i32, _vp, _vp, _vp, _vp]),
    "fathom_greedy_budgets": (ctypes.c_int, [_i32, _i32, _vp, _i32, _i32, _i32, _vp]),
    "fathom_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Shape), ctypes.c_int]),
    "fathom_last_error": (ctypes.c_char_p, []),
    "fathom_version": (ctypes.c_char_p, []),
    "fathom_debug_status": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p]),
}


class FathomError(RuntimeError):
    def __init__(self, name, status, msg):
        super().__init__(f"{name} failed with status {status}: {msg}")
        self.status = status


_lib = None


def lib():
    """Load libfathom.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfathom is not built ({LIB_PATH} missing): run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _call(name, *args):
    rc = getattr(lib(), name)(*args)
    if rc != 0:
        raise FathomError(name, rc, lib().fathom_last_error().decode())
    return rc


def _p(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtypes, shape=None, dev=True, min_numel=None):
    """Dtype, shape (exact), size (at least min_numel elements: the library sees only
    a pointer, so a shorter tensor would be read or written past its end),
    contiguity, and memory the GPU can reach, in that order."""
    if t is None:
        raise ValueError(f"{name} is required")
    if dtypes and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs at least {min_numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dev and not _reachable(t):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    return t


def _reachable(t) -> bool:
    """Memory the GPU can load from and store to: device memory or pinned host memory."""
    return t.is_cuda or t.is_pinned()


def _check_out(t, name, dtypes, min_numel):
    """A caller-provided output (None: the binding allocates it)."""
    if t is not None:
        _check(t, name, dtypes, min_numel=min_numel)
    return t


def _store_words(shape: Shape) -> int:
    """Elements of a bit-plane store [units][D][4][cap blocks]."""
    return shape.units * shape.D * 4 * nblocks(shape.cap)


def _store_scales(shape: Shape) -> int:
    """Elements of the store's scales [units][D][cap blocks]."""
    return shape.units * shape.D * nblocks(shape.cap)


def _rows(shape: Shape) -> int:
    """Elements of per-unit rows [units][cap][D]."""
    return shape.units * shape.cap * shape.D


def make_shape(units, n, D=128, G=4, k=1, n_sink=4, n_recent=32, n_cap=0, scan_ctas_per_sm=0) -> Shape:
    return Shape(units, n, D, G, k, n_sink, n_recent, n_cap, scan_ctas_per_sm)


def nblocks(n: int) -> int:
    return (n + 63) // 64


def version() -> str:
    return lib().fathom_version().decode()


def workspace_size(shape: Shape, which: int) -> int:
    return int(lib().fathom_workspace_size(ctypes.byref(shape), which))


def alloc_workspace(shape: Shape, which: int, device="cuda") -> torch.Tensor:
    nbytes = workspace_size(shape, which)
    if nbytes == 0:
        raise FathomError("fathom_workspace_size", 1, lib().fathom_last_error().decode())
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ calls
def fathom_calibrate(calib, mean=None, var=None, stream=None):
    """calib [U][m][D] fp32 -> (mean [U][D], var [U][D]) fp32 (ddof = 1)."""
    _check(calib, "calib", (torch.float32,))
    if calib.dim() != 3:
        raise ValueError(f"calib: shape {tuple(calib.shape)} is not [units][m][D]")
    U, m, D = calib.shape
    _check_out(mean, "mean", (torch.float32,), U * D)
    _check_out(var, "var", (torch.float32,), U * D)
    if var is None:
        var = torch.empty(U, D, dtype=torch.float32, device=calib.device)
    if mean is None:
        mean = torch.empty(U, D, dtype=torch.float32, device=calib.device)
    _call("fathom_calibrate", U, m, D, _p(calib), _p(mean), _p(var), _stream(stream))
    return mean, var


def fathom_calibrate_klt(calib, mean=None, V=None, lam=None, stream=None):
    """calib [groups][m][D] fp32 -> (mean [groups][D] fp64, V [groups][D][D] fp64 (eigenvectors
    as columns, eigenvalues descending), lambda [groups][D] fp32)."""
    _check(calib, "calib", (torch.float32,))
    if calib.dim() != 3:
        raise ValueError(f"calib: shape {tuple(calib.shape)} is not [groups][m][D]")
    Gr, m, D = calib.shape
    dev = calib.device
    _check_out(mean, "mean", (torch.float64,), Gr * D)
    _check_out(V, "V", (torch.float64,), Gr * D * D)
    _check_out(lam, "lam", (torch.float32,), Gr * D)
    if mean is None:
        mean = torch.empty(Gr, D, dtype=torch.float64, device=dev)
    if V is None:
        V = torch.empty(Gr, D, D, dtype=torch.float64, device=dev)
    if lam is None:
        lam = torch.empty(Gr, D, dtype=torch.float32, device=dev)
    _call("fathom_calibrate_klt", Gr, m, D, _p(calib), _p(mean), _p(V), _p(lam), _stream(stream))
    return mean, V, lam


def fathom_rotate_keys(shape: Shape, keys, groups, mean, V, out=None, stream=None):
    """keys [U][n][D] fp32 or bf16 -> (k - mu_g) V_g [U][n][D] fp32, g = u % groups."""
    _check(keys, "keys", (torch.float32, torch.bfloat16, torch.int16), min_numel=_rows(shape))
    _check(mean, "mean", (torch.float64,), (groups, shape.D))
    _check(V, "V", (torch.float64,), (groups, shape.D, shape.D))
    _check_out(out, "out", (torch.float32,), _rows(shape))
    dt = F32 if keys.dtype == torch.float32 else BF16
    if out is None:
        out = torch.empty(shape.units, shape.cap, shape.D, dtype=torch.float32, device=keys.device)
    _call("fathom_rotate_keys", ctypes.byref(shape), _p(keys), dt, int(groups), _p(mean), _p(V), _p(out),
          _stream(stream))
    return out


def fathom_rotate_query(shape: Shape, q, groups, V, out=None, stream=None):
    """q [U][G][D] fp32 -> q V_g [U][G][D] fp32, g = u % groups."""
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(V, "V", (torch.float64,), (groups, shape.D, shape.D))
    _check_out(out, "out", (torch.float32,), shape.units * shape.G * shape.D)
    if out is None:
        out = torch.empty_like(q)
    _call("fathom_rotate_query", ctypes.byref(shape), _p(q), int(groups), _p(V), _p(out), _stream(stream))
    return out


def fathom_quantize_pack(shape: Shape, keys, planes=None, scales=None, stream=None):
    """keys [U][n][D] fp32 or bf16 -> planes [U][D][4][nb] (int64 storage of u64),
    scales [U][D][nb] (int16 storage of fp16 bits)."""
    _check(keys, "keys", (torch.float32, torch.bfloat16, torch.int16), min_numel=_rows(shape))
    _check_out(planes, "planes", (torch.int64,), _store_words(shape))
    _check_out(scales, "scales", (torch.int16,), _store_scales(shape))
    dt = F32 if keys.dtype == torch.float32 else BF16
    nb = nblocks(shape.cap)
    dev = keys.device
    if planes is None:
        planes = torch.empty(shape.units, shape.D, 4, nb, dtype=torch.int64, device=dev)
    if scales is None:
        scales = torch.empty(shape.units, shape.D, nb, dtype=torch.int16, device=dev)
    _call("fathom_quantize_pack", ctypes.byref(shape), _p(keys), dt, _p(planes), _p(scales),
          _stream(stream))
    return planes, scales


def fathom_append_block(shape: Shape, keys, block, count, planes, scales, stream=None):
    """Quantise block `block` (its first `count` tokens) of every unit of the key rows
    keys [U][cap][D] (fp32 or bf16) into the store planes [U][D][4][cap blocks],
    scales [U][D][cap blocks], in place."""
    _check(keys, "keys", (torch.float32, torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(planes, "planes", (torch.int64,), (shape.units, shape.D, 4, nblocks(shape.cap)))
    _check(scales, "scales", (torch.int16,), (shape.units, shape.D, nblocks(shape.cap)))
    dt = F32 if keys.dtype == torch.float32 else BF16
    _call("fathom_append_block", ctypes.byref(shape), _p(keys), dt, int(block), int(count), _p(planes), _p(scales),
          _stream(stream))
    return planes, scales


def fathom_plan(shape: Shape, q, var, budget, bracket=None, depth=None, theta=None, runs=None,
                stream=None, want_theta=True):
    """-> depth [U][D] u8, theta [U] f64 (None when want_theta is False: the call
    then passes no theta buffer and the depths and runs are the same), runs
    [U][D][6] (int32 storage of u32)."""
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(var, "var", (torch.float32,), (shape.units, shape.D))
    _check(budget, "budget", (torch.int32,), (shape.units,))
    if bracket is not None:
        _check(bracket, "bracket", (torch.float64,), (shape.units, 2))
    _check_out(depth, "depth", (torch.uint8,), shape.units * shape.D)
    _check_out(theta, "theta", (torch.float64,), shape.units)
    _check_out(runs, "runs", (torch.int32,), shape.units * shape.D * 6)
    dev = q.device
    if depth is None:
        depth = torch.empty(shape.units, shape.D, dtype=torch.uint8, device=dev)
    if not want_theta:
        theta = None
    elif theta is None:
        theta = torch.empty(shape.units, dtype=torch.float64, device=dev)
    if runs is None:
        runs = torch.empty(shape.units, shape.D, 6, dtype=torch.int32, device=dev)
    _call("fathom_plan", ctypes.byref(shape), _p(q), _p(var), _p(budget), _p(bracket), _p(depth),
          _p(theta), _p(runs), _stream(stream))
    return depth, theta, runs


def fathom_plan_fixed(shape: Shape, q, var, n_channels, depth_each, depth=None, runs=None,
                      stream=None):
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(var, "var", (torch.float32,), (shape.units, shape.D))
    _check_out(depth, "depth", (torch.uint8,), shape.units * shape.D)
    _check_out(runs, "runs", (torch.int32,), shape.units * shape.D * 6)
    dev = q.device
    if depth is None:
        depth = torch.empty(shape.units, shape.D, dtype=torch.uint8, device=dev)
    if runs is None:
        runs = torch.empty(shape.units, shape.D, 6, dtype=torch.int32, device=dev)
    _call("fathom_plan_fixed", ctypes.byref(shape), _p(q), _p(var), int(n_channels), int(depth_each),
          _p(depth), _p(runs), _stream(stream))
    return depth, runs


def fathom_gather(shape: Shape, store_planes, store_scales, runs, stage_planes, stage_scales,
                  stream=None):
    """stage_planes [U][W] int64, stage_scales [U][S] int16 (per-unit strides W, S)."""
    _check(store_planes, "store_planes", (torch.int64,), min_numel=_store_words(shape))
    _check(store_scales, "store_scales", (torch.int16,), min_numel=_store_scales(shape))
    _check(runs, "runs", (torch.int32,), (shape.units, shape.D, 6))
    W = stage_planes.shape[-1] if stage_planes is not None and stage_planes.dim() else 0
    S = stage_scales.shape[-1] if stage_scales is not None and stage_scales.dim() else 0
    _check(stage_planes, "stage_planes", (torch.int64,), min_numel=shape.units * W)
    _check(stage_scales, "stage_scales", (torch.int16,), min_numel=shape.units * S)
    _call("fathom_gather", ctypes.byref(shape), _p(store_planes), _p(store_scales), _p(runs),
          _p(stage_planes), _p(stage_scales), W, S, _stream(stream))
    return stage_planes, stage_scales


def fathom_scan_topk(shape: Shape, planes, scales, runs, q, workspace, source=SRC_STORE,
                     topk_idx=None, topk_score=None, scores=None, stream=None):
    """-> topk_idx [U][G][k] int32 ascending, topk_score [U][G][k] fp32 (scores, if given,
    receives every token's score [U][G][n])."""
    if source == SRC_STAGING:      # [units][W] and [units][S]: the last dimension is the per-unit stride
        W = planes.shape[-1] if planes is not None and planes.dim() else 0
        S = scales.shape[-1] if scales is not None and scales.dim() else 0
        need_p, need_s = shape.units * W, shape.units * S
    else:
        W = S = 0
        need_p, need_s = _store_words(shape), _store_scales(shape)
    _check(planes, "planes", (torch.int64,), min_numel=need_p)
    _check(scales, "scales", (torch.int16,), min_numel=need_s)
    _check(runs, "runs", (torch.int32,), (shape.units, shape.D, 6))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(workspace, "workspace", (torch.uint8,))
    _check_out(topk_idx, "topk_idx", (torch.int32,), shape.units * shape.G * shape.k)
    _check_out(topk_score, "topk_score", (torch.float32,), shape.units * shape.G * shape.k)
    dev = q.device
    if topk_idx is None:
        topk_idx = torch.empty(shape.units, shape.G, shape.k, dtype=torch.int32, device=dev)
    if topk_score is None:
        topk_score = torch.empty(shape.units, shape.G, shape.k, dtype=torch.float32, device=dev)
    if scores is not None:
        _check(scores, "scores", (torch.float32,), (shape.units, shape.G, shape.n))
    _call("fathom_scan_topk", ctypes.byref(shape), _p(planes), _p(scales), int(source), W, S,
          _p(runs), _p(q), _p(topk_idx), _p(topk_score), _p(scores), _p(workspace),
          workspace.numel(), _stream(stream))
    return topk_idx, topk_score


def _scan_inputs(shape, planes, scales, runs, q, workspace, source):
    if source == SRC_STAGING:
        W = planes.shape[-1] if planes is not None and planes.dim() else 0
        S = scales.shape[-1] if scales is not None and scales.dim() else 0
        need_p, need_s = shape.units * W, shape.units * S
    else:
        W = S = 0
        need_p, need_s = _store_words(shape), _store_scales(shape)
    _check(planes, "planes", (torch.int64,), min_numel=need_p)
    _check(scales, "scales", (torch.int16,), min_numel=need_s)
    _check(runs, "runs", (torch.int32,), (shape.units, shape.D, 6))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(workspace, "workspace", (torch.uint8,))
    return W, S


def fathom_scan(shape: Shape, planes, scales, runs, q, workspace, source=SRC_STORE, scores=None, stream=None):
    """The scan half of fathom_scan_topk: candidate lists in the workspace (scores, if
    given, receives every token's score [U][G][n])."""
    W, S = _scan_inputs(shape, planes, scales, runs, q, workspace, source)
    if scores is not None:
        _check(scores, "scores", (torch.float32,), (shape.units, shape.G, shape.n))
    _call("fathom_scan", ctypes.byref(shape), _p(planes), _p(scales), int(source), W, S, _p(runs), _p(q),
          _p(scores), _p(workspace), workspace.numel(), _stream(stream))


def fathom_select(shape: Shape, planes, scales, runs, q, workspace, source=SRC_STORE, topk_idx=None,
                  topk_score=None, stream=None):
    """The selection half: -> topk_idx [U][G][k] int32 ascending, topk_score [U][G][k] fp32."""
    W, S = _scan_inputs(shape, planes, scales, runs, q, workspace, source)
    _check_out(topk_idx, "topk_idx", (torch.int32,), shape.units * shape.G * shape.k)
    _check_out(topk_score, "topk_score", (torch.float32,), shape.units * shape.G * shape.k)
    if topk_idx is None:
        topk_idx = torch.empty(shape.units, shape.G, shape.k, dtype=torch.int32, device=q.device)
    if topk_score is None:
        topk_score = torch.empty(shape.units, shape.G, shape.k, dtype=torch.float32, device=q.device)
    _call("fathom_select", ctypes.byref(shape), _p(planes), _p(scales), int(source), W, S, _p(runs), _p(q),
          _p(topk_idx), _p(topk_score), _p(workspace), workspace.numel(), _stream(stream))
    return topk_idx, topk_score


def fathom_exact_topk(shape: Shape, k_rows, q, workspace, topk_idx=None, topk_score=None, scores=None,
                      stream=None):
    """Fidelity reference: the kept set with every token scored exactly, q . k
    over all D channels of its bf16 row.  k_rows [U][cap][D] bf16 -> topk_idx
    [U][G][k] int32 ascending, topk_score [U][G][k] fp32 (workspace of kind
    WS_SCAN_TOPK)."""
    _check(k_rows, "k_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(workspace, "workspace", (torch.uint8,))
    _check_out(topk_idx, "topk_idx", (torch.int32,), shape.units * shape.G * shape.k)
    _check_out(topk_score, "topk_score", (torch.float32,), shape.units * shape.G * shape.k)
    dev = q.device
    if topk_idx is None:
        topk_idx = torch.empty(shape.units, shape.G, shape.k, dtype=torch.int32, device=dev)
    if topk_score is None:
        topk_score = torch.empty(shape.units, shape.G, shape.k, dtype=torch.float32, device=dev)
    if scores is not None:
        _check(scores, "scores", (torch.float32,), (shape.units, shape.G, shape.n))
    _call("fathom_exact_topk", ctypes.byref(shape), _p(k_rows), _p(q), _p(topk_idx), _p(topk_score),
          _p(scores), _p(workspace), workspace.numel(), _stream(stream))
    return topk_idx, topk_score


def fathom_dense_attn(shape: Shape, k_rows, v_rows, q, workspace, out=None, stream=None):
    """Fidelity reference: attention of every head over all n tokens.
    k_rows, v_rows [U][cap][D] bf16 -> out [U][G][D] fp32 (workspace of kind
    WS_DENSE_ATTN)."""
    _check(k_rows, "k_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(v_rows, "v_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(workspace, "workspace", (torch.uint8,))
    _check_out(out, "out", (torch.float32,), shape.units * shape.G * shape.D)
    if out is None:
        out = torch.empty(shape.units, shape.G, shape.D, dtype=torch.float32, device=q.device)
    _call("fathom_dense_attn", ctypes.byref(shape), _p(k_rows), _p(v_rows), _p(q), _p(out),
          _p(workspace), workspace.numel(), _stream(stream))
    return out


def fathom_klt_online(shape: Shape, k_rows, workspace=None, mean=None, V=None, lam=None, stream=None):
    """Per-unit rotated basis from the unit's own key rows [U][cap][D] bf16 ->
    (mean [U][D] f64, V [U][D][D] f64, lambda [U][D] f32)."""
    _check(k_rows, "k_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check_out(mean, "mean", (torch.float64,), shape.units * shape.D)
    _check_out(V, "V", (torch.float64,), shape.units * shape.D * shape.D)
    _check_out(lam, "lam", (torch.float32,), shape.units * shape.D)
    dev = "cuda"
    if workspace is None:
        workspace = alloc_workspace(shape, WS_KLT_ONLINE, device=dev)
    _check(workspace, "workspace", (torch.uint8,))
    U, D = shape.units, shape.D
    if mean is None:
        mean = torch.empty(U, D, dtype=torch.float64, device=dev)
    if V is None:
        V = torch.empty(U, D, D, dtype=torch.float64, device=dev)
    if lam is None:
        lam = torch.empty(U, D, dtype=torch.float32, device=dev)
    _call("fathom_klt_online", ctypes.byref(shape), _p(k_rows), _p(mean), _p(V), _p(lam), _p(workspace),
          workspace.numel(), _stream(stream))
    return mean, V, lam


def fathom_rel_err(a, ref, err=None, stream=None):
    """a, ref [..., D] fp32 (device) -> err [...] fp64: ||a - ref|| / ||ref|| per row."""
    _check(a, "a", (torch.float32,))
    _check(ref, "ref", (torch.float32,), tuple(a.shape))
    D = a.shape[-1]
    rows = a.numel() // D if D else 0
    if err is None:
        err = torch.empty(a.shape[:-1], dtype=torch.float64, device=a.device)
    _check(err, "err", (torch.float64,), tuple(a.shape[:-1]))
    _call("fathom_rel_err", rows, D, _p(a), _p(ref), _p(err), _stream(stream))
    return err


def fathom_set_overlap(a, b, count=None, stream=None):
    """a, b [..., k] int32 ascending (device) -> count [...] int32: shared indices per row."""
    _check(a, "a", (torch.int32,))
    _check(b, "b", (torch.int32,), tuple(a.shape))
    k = a.shape[-1]
    rows = a.numel() // k if k else 0
    if count is None:
        count = torch.empty(a.shape[:-1], dtype=torch.int32, device=a.device)
    _check(count, "count", (torch.int32,), tuple(a.shape[:-1]))
    _call("fathom_set_overlap", rows, k, _p(a), _p(b), _p(count), _stream(stream))
    return count


def fathom_greedy_budgets(err, b_min, step, b_mean):
    """err [layers][levels] (host array-like, fp64) -> budgets [layers] (numpy int32)."""
    import numpy as np
    e = np.ascontiguousarray(np.asarray(err, dtype=np.float64))
    if e.ndim != 2:
        raise ValueError("err must be [layers][levels]")
    out = np.zeros(e.shape[0], dtype=np.int32)
    _call("fathom_greedy_budgets", e.shape[0], e.shape[1], e.ctypes.data, int(b_min), int(step), int(b_mean),
          out.ctypes.data)
    return out


def fathom_sparse_attn_planes(shape: Shape, planes, scales, v_rows, q, topk_idx, workspace, out=None,
                              stream=None):
    """Sparse attention with the winners' keys rebuilt from the store's four planes.
    planes [U][D][4][cb], scales [U][D][cb], v_rows [U][cap][D] bf16 -> out [U][G][D] fp32."""
    cb = nblocks(shape.cap)
    _check(planes, "planes", (torch.int64,), (shape.units, shape.D, 4, cb))
    _check(scales, "scales", (torch.int16,), (shape.units, shape.D, cb))
    _check(v_rows, "v_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(topk_idx, "topk_idx", (torch.int32,), (shape.units, shape.G, shape.k))
    _check(workspace, "workspace", (torch.uint8,))
    _check_out(out, "out", (torch.float32,), shape.units * shape.G * shape.D)
    if out is None:
        out = torch.empty(shape.units, shape.G, shape.D, dtype=torch.float32, device=q.device)
    _call("fathom_sparse_attn_planes", ctypes.byref(shape), _p(planes), _p(scales), _p(v_rows), _p(q),
          _p(topk_idx), _p(out), _p(workspace), workspace.numel(), _stream(stream))
    return out


def fathom_sparse_attn_noalloc(shape: Shape, k_rows, v_rows, q, topk_idx, out, stream=None):
    """fathom_sparse_attn with the library's own fixed scratch (no workspace, no
    allocation inside the call): for callers that may not allocate device memory.
    `out` [U][G][D] fp32 must be provided by the caller."""
    _check(k_rows, "k_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(v_rows, "v_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(topk_idx, "topk_idx", (torch.int32,), (shape.units, shape.G, shape.k))
    _check(out, "out", (torch.float32,), (shape.units, shape.G, shape.D))
    _call("fathom_sparse_attn_noalloc", ctypes.byref(shape), _p(k_rows), _p(v_rows), _p(q),
          _p(topk_idx), _p(out), _stream(stream))
    return out


def fathom_sparse_attn(shape: Shape, k_rows, v_rows, q, topk_idx, workspace, out=None, stream=None):
    """k_rows, v_rows [U][n][D] bf16 (device or pinned host) -> out [U][G][D] fp32."""
    _check(k_rows, "k_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(v_rows, "v_rows", (torch.bfloat16, torch.int16), (shape.units, shape.cap, shape.D))
    _check(q, "q", (torch.float32,), (shape.units, shape.G, shape.D))
    _check(topk_idx, "topk_idx", (torch.int32,), (shape.units, shape.G, shape.k))
    _check(workspace, "workspace", (torch.uint8,))
    _check_out(out, "out", (torch.float32,), shape.units * shape.G * shape.D)
    if out is None:
        out = torch.empty(shape.units, shape.G, shape.D, dtype=torch.float32, device=q.device)
    _call("fathom_sparse_attn", ctypes.byref(shape), _p(k_rows), _p(v_rows), _p(q), _p(topk_idx),
          _p(out), _p(workspace), workspace.numel(), _stream(stream))
    return out


# ------------------------------------------------------- prompts and paged caches
_ROW_TYPES = {torch.bfloat16: BF16, torch.float16: F16}


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_NO_CONTEXT = contextlib.nullcontext()


def _on(stream, tensors):
    """(context, stream handle) of a call on these tensors: their device is made current
    (one device: the library launches on the current one) and, when a stream is given,
    that stream, so that outputs allocated inside belong to the stream that writes them."""
    device = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != device and d >= 0:
                if device >= 0:
                    raise ValueError(f"tensors on several devices: cuda:{device} and cuda:{d}")
                device = d
    if stream is None:
        if device < 0:
            return _NO_CONTEXT, _stream(None)
        if device == _current_device():
            return _NO_CONTEXT, _raw_stream(device) if _raw_stream else _stream(None)
        with torch.cuda.device(device):
            return torch.cuda.device(device), _stream(None)
    if device >= 0 and stream.device_index != device:
        raise ValueError(f"stream on cuda:{stream.device_index}, tensors on cuda:{device}")
    return torch.cuda.stream(stream), _stream(stream)


def _check_strided(t, name, dtypes, shape, pinned=False):
    """A tensor of these sizes whose last axis is contiguous, the others strided as
    they are; every element behind its pointer lies in the tensor's storage.  Device
    memory (pinned: or pinned host memory)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if not (_reachable(t) if pinned else _on_device(t)):
        raise ValueError(f"{name} must be a CUDA tensor" + (" or pinned host memory" if pinned else ""))
    return t


def _on_device(t) -> bool:
    return t.is_cuda


def _ok(t, dtype, shape):
    """A contiguous CUDA tensor of this type and these sizes (the common case, decided in
    one expression; anything else goes through the checks that name what is wrong)."""
    return t is not None and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()


def _fit32(**counts):
    """The library's counts are 32-bit, and ctypes would cut a larger one off without a word."""
    for name, x in counts.items():
        if not -(1 << 31) <= x < 1 << 31:
            raise ValueError(f"{name}: {x} does not fit 32 bits")


def fathom_prefill_attn(q, k, v, cu_q, cu_k=None, out=None, lse=None, want_lse=False, stream=None):
    """Causal attention of packed prompts (or of their next chunks): q [Tq][heads][D],
    k, v [Tk][kv_heads][D] bf16 or fp16, any strides with the last axis contiguous;
    cu_q, cu_k [seqs + 1] int32 (cu_k None: cu_q, whole prompts).  -> (out [Tq][heads][D]
    of q's type, lse [Tq][heads] fp32 or None; rows behind cu_q[-1] are not written)."""
    if q is None or q.dim() != 3:
        raise ValueError("q: expected [tokens][heads][D]")
    if k is None or k.dim() != 3:
        raise ValueError("k: expected [tokens][kv_heads][D]")
    Tq, H, D = q.shape
    Tk, Hkv, _ = k.shape
    dt = q.dtype
    if Tq >> 31 or Tk >> 31:
        _fit32(query_tokens=Tq, key_tokens=Tk)
    (qt, qh, qc), (kt, kh, kc) = q.stride(), k.stride()
    if not (dt in _ROW_TYPES and qc == 1 and q.is_cuda):
        _check_strided(q, "q", _ROW_TYPES, (Tq, H, D))
    if not (k.dtype is dt and k.shape[2] == D and kc == 1 and k.is_cuda):
        _check_strided(k, "k", (dt,), (Tk, Hkv, D))
    if v is None or not (v.dtype is dt and v.shape == (Tk, Hkv, D) and v.stride(2) == 1 and v.is_cuda):
        _check_strided(v, "v", (dt,), (Tk, Hkv, D))
    vt, vh, _ = v.stride()
    if cu_k is None:
        cu_k = cu_q
    _check(cu_q, "cu_q", (torch.int32,))
    if cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError(f"cu_q: shape {tuple(cu_q.shape)} is not [seqs + 1]")
    if not _ok(cu_k, torch.int32, cu_q.shape):
        _check(cu_k, "cu_k", (torch.int32,), tuple(cu_q.shape))
    if out is not None:
        _check_strided(out, "out", (dt,), (Tq, H, D))
    if lse is not None:
        _check(lse, "lse", (torch.float32,), (Tq, H))
    context, handle = _on(stream, (q, k, v, cu_q, cu_k, out, lse))
    with context:
        if out is None:
            out = torch.empty((Tq, H, D), dtype=dt, device=q.device)
        if lse is None and want_lse:
            lse = torch.empty((Tq, H), dtype=torch.float32, device=q.device)
        ot, oh, _ = out.stride()
        p = Prompts(cu_q.shape[0] - 1, H, Hkv, D, _ROW_TYPES[dt], Tq, Tk, qt, qh, kt, kh, vt, vh, ot, oh)
        _call("fathom_prefill_attn", p, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
              out.data_ptr(), lse.data_ptr() if lse is not None else None, handle)
    return out, lse


def make_pages(k_pages, page_table) -> Pages:
    """The layout of a paged cache: k_pages a [pages][kv_heads][page_tokens][D] view of
    bf16 or fp16 rows (any strides, the last axis contiguous; v_pages must have the
    same), page_table [seqs][max_pages] int32."""
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages: expected [pages][kv_heads][page_tokens][D], page_table: [seqs][max_pages]")
    if k_pages.dtype not in _ROW_TYPES:
        raise TypeError(f"k_pages: dtype {k_pages.dtype} not in {tuple(_ROW_TYPES)}")
    (n, H, P, D), (seqs, per) = k_pages.shape, page_table.shape
    if (n | P | per) >> 31:
        _fit32(pages=n, page_tokens=P, max_pages=per)
    sn, sh, sp, _ = k_pages.stride()
    return Pages(seqs, H, D, _ROW_TYPES[k_pages.dtype], P, n, per, sn, sh, sp)


def rows_as_pages(rows, kv_heads, page_tokens=64, device=None):
    """Rows [units][C][D] of the other calls (units packed sequence, KV head; page_tokens
    divides C) seen as a paged cache: (view [pages][kv_heads][page_tokens][D], page_table
    [seqs][C / page_tokens] on `device`, the rows' by default).  The view shares the
    rows' memory."""
    U, C, D = rows.shape
    if not rows.is_contiguous() or U % kv_heads or C % page_tokens:
        raise ValueError("rows: contiguous [units][C][D], kv_heads dividing units and page_tokens dividing C")
    seqs, per = U // kv_heads, C // page_tokens
    # page number x page_tokens * D elements; a sequence's pages are those of its first head
    count = (seqs - 1) * kv_heads * per + per
    view = rows.as_strided((count, kv_heads, page_tokens, D), (page_tokens * D, C * D, D, 1))
    table = (torch.arange(seqs, dtype=torch.int32)[:, None] * (kv_heads * per) +
             torch.arange(per, dtype=torch.int32)[None, :]).to(device or rows.device)
    return view, table


def _check_cache(pages, k_pages, v_pages, page_table):
    """-> (type of the rows, sequences, KV heads, D, tokens a table row can name)."""
    seqs, H, D, dt, P, n, per = (pages.seqs, pages.kv_heads, pages.D, pages.dtype, pages.page_tokens, pages.num_pages,
                                 pages.max_pages)
    dtype = torch.bfloat16 if dt == BF16 else torch.float16
    shape, stride = (n, H, P, D), (pages.page_stride, pages.head_stride, pages.token_stride, 1)
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t is not None and t.dtype is dtype and t.shape == shape and t.stride() == stride and t.is_cuda:
            continue
        _check_strided(t, name, (dtype,), shape, pinned=True)
        if any(a > 1 and x != y for a, x, y in zip(shape, t.stride(), stride)):
            raise ValueError(f"{name}: strides {t.stride()[:3]} are not those of pages")
    if not _ok(page_table, torch.int32, (seqs, per)):
        _check(page_table, "page_table", (torch.int32,), (seqs, per))
    return dtype, seqs, H, D, per * P


def paged_workspace_size(pages: Pages, G: int, mass=False) -> int:
    return int(lib().fathom_paged_workspace_size(ctypes.byref(pages), int(G), int(bool(mass))))


def alloc_paged_workspace(pages: Pages, G=4, mass=False, device="cuda") -> torch.Tensor:
    """Workspace of fathom_paged_attn (mass: also large enough for calls with it).  One that is large enough for
    several calls of different sizes serves them in any order."""
    nbytes = paged_workspace_size(pages, G, mass)
    if nbytes == 0:
        raise FathomError("fathom_paged_workspace_size", 1, lib().fathom_last_error().decode())
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def fathom_paged_append(pages: Pages, k_pages, v_pages, page_table, k_new, v_new, start, cu_new=None, stream=None):
    """Write new rows k_new, v_new [T][kv_heads][D] (strided alike, the last axis contiguous)
    into the cache, in place: token i of sequence s at position start[s] + i.  start [seqs]
    int32; cu_new [seqs + 1] int32, or None: one token per sequence."""
    dtype, seqs, H, D, _ = _check_cache(pages, k_pages, v_pages, page_table)
    if k_new is None or k_new.dim() != 3:
        raise ValueError("k_new: expected [tokens][kv_heads][D]")
    T = k_new.shape[0]
    if T >> 31:
        _fit32(new_tokens=T)
    _check_strided(k_new, "k_new", (dtype,), (T, H, D))
    _check_strided(v_new, "v_new", (dtype,), (T, H, D))
    stride = k_new.stride()
    if stride != v_new.stride() and any(a > 1 and x != y for a, x, y in zip((T, H), stride, v_new.stride())):
        raise ValueError("v_new: strides differ from k_new's")
    if not _ok(start, torch.int32, (seqs,)):
        _check(start, "start", (torch.int32,), (seqs,))
    if cu_new is not None:
        if not _ok(cu_new, torch.int32, (seqs + 1,)):
            _check(cu_new, "cu_new", (torch.int32,), (seqs + 1,))
    elif T != seqs:
        raise ValueError(f"k_new: {T} tokens for {seqs} sequences without cu_new")
    context, handle = _on(stream, (k_pages, v_pages, page_table, k_new, v_new, start, cu_new))
    with context:
        _call("fathom_paged_append", pages, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
              k_new.data_ptr(), v_new.data_ptr(), T, stride[0], stride[1], start.data_ptr(),
              cu_new.data_ptr() if cu_new is not None else None, handle)
    return k_pages, v_pages


def fathom_paged_attn(pages: Pages, q, k_pages, v_pages, page_table, lens, workspace, out=None, mass=None,
                      stream=None):
    """Decode attention over the cache: q [units][G][D] fp32, lens [seqs] int32 -> out
    [units][G][D] fp32.  mass [units][M] fp32, M >= pages.cap: each token's attention
    weights, summed over the G heads, are added to it (workspace allocated with mass)."""
    _, seqs, H, D, cap = _check_cache(pages, k_pages, v_pages, page_table)
    if q is None or q.dim() != 3:
        raise ValueError("q: expected [units][G][D]")
    G = q.shape[1]
    shape = (seqs * H, G, D)
    if not _ok(q, torch.float32, shape):
        _check(q, "q", (torch.float32,), shape)
    if not _ok(lens, torch.int32, (seqs,)):
        _check(lens, "lens", (torch.int32,), (seqs,))
    _check(workspace, "workspace", (torch.uint8,))
    if out is not None and not _ok(out, torch.float32, shape):
        _check(out, "out", (torch.float32,), shape)
    if mass is not None:
        _check_mass(mass, "mass", seqs * H, cap)
    context, handle = _on(stream, (q, k_pages, v_pages, page_table, lens, workspace, out, mass))
    with context:
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=q.device)
        _call("fathom_paged_attn", pages, G, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
              page_table.data_ptr(), lens.data_ptr(), out.data_ptr(), mass.data_ptr() if mass is not None else None,
              mass.shape[1] if mass is not None else 0, workspace.data_ptr(), workspace.numel(), handle)
    return out


def _check_mass(t, name, units, least):
    _check(t, name, (torch.float32,))
    if t.dim() != 2 or t.shape[0] != units or t.shape[1] < least:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not [{units}][at least {least}]")


def fathom_paged_evict(pages: Pages, k_pages, v_pages, page_table, lens, mass, keep, dst_table, n_sink=4,
                       n_recent=32, kept_idx=None, lens_out=None, mass_out=None, stream=None):
    """Cut every unit back to `keep` tokens by attention mass; the kept rows move, in order,
    to the pages of dst_table [seqs][pages] (page_table itself: in place).  -> (kept_idx
    [units][keep] int32, ascending and then -1, lens_out [seqs] int32, mass_out
    [units][M] fp32; mass_out None: mass itself, in place).  Mass behind the kept tokens
    is left as it was: set it to 0 before new tokens take those places."""
    _, seqs, H, _, cap = _check_cache(pages, k_pages, v_pages, page_table)
    keep, units = int(keep), seqs * H
    if not _ok(lens, torch.int32, (seqs,)):
        _check(lens, "lens", (torch.int32,), (seqs,))
    _check_mass(mass, "mass", units, cap)
    _check(dst_table, "dst_table", (torch.int32,))
    if dst_table.dim() != 2 or dst_table.shape[0] != seqs:
        raise ValueError(f"dst_table: shape {tuple(dst_table.shape)} is not [{seqs}][pages]")
    _fit32(keep=keep, n_sink=int(n_sink), n_recent=int(n_recent), dst_pages=dst_table.shape[1])
    if mass_out is None:
        mass_out = mass
    _check_mass(mass_out, "mass_out", units, keep)
    if kept_idx is not None:
        _check(kept_idx, "kept_idx", (torch.int32,), (units, keep))
    if lens_out is not None:
        _check(lens_out, "lens_out", (torch.int32,), (seqs,))
    context, handle = _on(stream, (k_pages, v_pages, page_table, lens, mass, dst_table, kept_idx, lens_out, mass_out))
    with context:
        if kept_idx is None:
            kept_idx = torch.empty((units, keep), dtype=torch.int32, device=mass.device)
        if lens_out is None:
            lens_out = torch.empty(seqs, dtype=torch.int32, device=mass.device)
        _call("fathom_paged_evict", pages, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
              lens.data_ptr(), mass.data_ptr(), mass.shape[1], keep, int(n_sink), int(n_recent), dst_table.data_ptr(),
              dst_table.shape[1], kept_idx.data_ptr(), lens_out.data_ptr(), mass_out.data_ptr(), mass_out.shape[1],
              handle)
    return kept_idx, lens_out, mass_out


# ------------------------------------------------------- position rotation and the 4-bit cache
_OUT_TYPES = {torch.float32: F32, **_ROW_TYPES}


def _rows_ok(t, dtype, shape):
    """Rows of this type and these sizes with a contiguous last axis on a GPU (the common case)."""
    return t is not None and t.dtype is dtype and t.shape == shape and t.stride(2) == 1 and t.is_cuda


def _check_rope(rope, positions, q, q_out, q_dtype, dtype, T, D):
    """-> the type of the rotated queries (None: there are none)."""
    if rope is None:
        if positions is not None or q is not None or q_out is not None or q_dtype is not None:
            raise ValueError("rope is required with positions, q, q_out or q_dtype")
        return None
    if not (rope.dtype is torch.float32 and rope.dim() == 2 and rope.is_cuda and rope.is_contiguous()):
        _check(rope, "rope", (torch.float32,))
        if rope.dim() != 2:
            raise ValueError(f"rope: shape {tuple(rope.shape)} is not [positions][rotated channels]")
        if not _on_device(rope):
            raise ValueError("rope must be a CUDA tensor")
    rows, rot = rope.shape
    if not 0 < rows < 1 << 31 or rot >> 31:
        raise ValueError(f"rope: {rows} positions of {rot} channels")
    if positions is not None and not _ok(positions, torch.int32, (T,)):
        _check(positions, "positions", (torch.int32,), (T,))
    if q is None:
        if q_out is not None or q_dtype is not None:
            raise ValueError("q is required with q_out or q_dtype")
        return None
    if q.dim() != 3:
        raise ValueError("q: expected [tokens][heads][D]")
    shape = (T, q.shape[1], D)
    if not _rows_ok(q, dtype, shape):
        _check_strided(q, "q", (dtype,), shape)
    if q_dtype is None:
        q_dtype = q_out.dtype if q_out is not None else dtype
    if q_dtype is not dtype and q_dtype is not torch.float32:
        raise TypeError(f"q_dtype: {q_dtype} is neither {dtype} nor torch.float32")
    if q_out is not None and not _rows_ok(q_out, q_dtype, shape):
        _check_strided(q_out, "q_out", (q_dtype,), shape)
    return q_dtype


def _make_rope(rope, positions, interleaved, q, q_out, q_dtype):
    """-> (the call's rotation or None, the rotated queries' place, allocated here unless given, or None)."""
    if rope is None:
        return None, None
    rows, rot = rope.shape
    at = positions.data_ptr() if positions is not None else None
    if q is None:
        return Rope(rope.data_ptr(), rows, rot, 1 if interleaved else 0, at), None
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q_dtype, device=q.device)
    (qt, qh, _), (ot, oh, _) = q.stride(), q_out.stride()
    return Rope(rope.data_ptr(), rows, rot, 1 if interleaved else 0, at, q.data_ptr(), q_out.data_ptr(), q.shape[1],
                _OUT_TYPES[q_dtype], qt, qh, ot, oh), q_out


def _check_new(k_new, v_new, start, cu_new, dtype, seqs, H, D):
    """-> (new tokens, their strides)."""
    if k_new is None or k_new.dim() != 3:
        raise ValueError("k_new: expected [tokens][kv_heads][D]")
    T = k_new.shape[0]
    if T >> 31:
        _fit32(new_tokens=T)
    shape, stride = (T, H, D), k_new.stride()
    if not (k_new.dtype is dtype and k_new.shape == shape and stride[2] == 1 and k_new.is_cuda):
        _check_strided(k_new, "k_new", (dtype,), shape)
    if v_new is None or not (v_new.dtype is dtype and v_new.shape == shape and v_new.stride() == stride and v_new.is_cuda):
        _check_strided(v_new, "v_new", (dtype,), shape)
    if stride != v_new.stride() and any(a > 1 and x != y for a, x, y in zip((T, H), stride, v_new.stride())):
        raise ValueError("v_new: strides differ from k_new's")
    if not _ok(start, torch.int32, (seqs,)):
        _check(start, "start", (torch.int32,), (seqs,))
    if cu_new is not None:
        if not _ok(cu_new, torch.int32, (seqs + 1,)):
            _check(cu_new, "cu_new", (torch.int32,), (seqs + 1,))
    elif T != seqs:
        raise ValueError(f"k_new: {T} tokens for {seqs} sequences without cu_new")
    return T, stride


def fathom_paged_append_rope(pages: Pages, k_pages, v_pages, page_table, k_new, v_new, start, rope, cu_new=None,
                             positions=None, interleaved=False, q=None, q_out=None, q_dtype=None, stream=None):
    """fathom_paged_append with the position rotation: rope [positions][rot] fp32 holds cos, then sin, of
    each position's rot / 2 angles; keys, and queries q [T][heads][D] if given, are rotated on the way.
    positions [T] int32 (None: a token's place in its sequence).  -> (k_pages, v_pages, rotated queries
    of q_dtype, the rows' type or torch.float32, or None)."""
    dtype, seqs, H, D, _ = _check_cache(pages, k_pages, v_pages, page_table)
    T, stride = _check_new(k_new, v_new, start, cu_new, dtype, seqs, H, D)
    if rope is None:
        raise ValueError("rope is required")
    q_dtype = _check_rope(rope, positions, q, q_out, q_dtype, dtype, T, D)
    context, handle = _on(stream, (k_pages, v_pages, page_table, k_new, v_new, start, cu_new, rope, positions, q, q_out))
    with context:
        r, q_out = _make_rope(rope, positions, interleaved, q, q_out, q_dtype)
        _call("fathom_paged_append_rope", pages, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
              k_new.data_ptr(), v_new.data_ptr(), T, stride[0], stride[1], start.data_ptr(),
              cu_new.data_ptr() if cu_new is not None else None, r, handle)
    return k_pages, v_pages, q_out


def alloc_nibble_pages(num_pages, kv_heads, page_tokens, D, device="cuda") -> torch.Tensor:
    """Pages of a 4-bit cache, all zeros (values 0): [num_pages][kv_heads][bytes of a page]."""
    return torch.zeros(num_pages, kv_heads, page_tokens // 16 * 18 * D, dtype=torch.uint8, device=device)


def make_nibble_pages(kv_pages, page_table, D) -> NibblePages:
    """The layout of a 4-bit cache: kv_pages uint8 [pages][kv_heads][bytes of a page, 18 D per 16
    tokens] (pages and heads strided as they are), page_table [seqs][max_pages] int32."""
    if kv_pages.dim() != 3 or page_table.dim() != 2:
        raise ValueError("kv_pages: expected [pages][kv_heads][bytes], page_table: [seqs][max_pages]")
    if kv_pages.dtype != torch.uint8:
        raise TypeError(f"kv_pages: dtype {kv_pages.dtype} is not torch.uint8")
    (n, H, size), (seqs, per) = kv_pages.shape, page_table.shape
    if D < 1 or size == 0 or size % (18 * D):
        raise ValueError(f"kv_pages: {size} bytes are no blocks of 18 * {D}")
    tokens = size // (18 * D) * 16
    if (n | tokens | per) >> 31:
        _fit32(pages=n, page_tokens=tokens, max_pages=per)
    sn, sh, _ = kv_pages.stride()
    return NibblePages(seqs, H, D, tokens, n, per, sn, sh)


def _check_nibble(pages, kv_pages, page_table):
    """-> (sequences, KV heads, D)."""
    seqs, H, D, P, n, per = pages.seqs, pages.kv_heads, pages.D, pages.page_tokens, pages.num_pages, pages.max_pages
    shape, stride = (n, H, P // 16 * 18 * D), (pages.page_stride, pages.head_stride, 1)
    if not (kv_pages is not None and kv_pages.dtype is torch.uint8 and kv_pages.shape == shape
            and kv_pages.stride() == stride and kv_pages.is_cuda):
        _check_strided(kv_pages, "kv_pages", (torch.uint8,), shape)
        if any(a > 1 and x != y for a, x, y in zip(shape, kv_pages.stride(), stride)):
            raise ValueError(f"kv_pages: strides {kv_pages.stride()[:2]} are not those of pages")
    if not _ok(page_table, torch.int32, (seqs, per)):
        _check(page_table, "page_table", (torch.int32,), (seqs, per))
    return seqs, H, D


def fathom_nibble_append(pages: NibblePages, kv_pages, page_table, k_new, v_new, start, cu_new=None, rope=None,
                         positions=None, interleaved=False, q=None, q_out=None, q_dtype=None, stream=None):
    """Write new rows k_new, v_new [T][kv_heads][D] (bf16 or fp16) into a 4-bit cache, in place, keys and
    queries rotated on the way if rope is given; tokens, rotation and queries as in
    fathom_paged_append_rope.  -> (kv_pages, rotated queries or None)."""
    seqs, H, D = _check_nibble(pages, kv_pages, page_table)
    dtype = k_new.dtype if k_new is not None else None
    if dtype not in _ROW_TYPES:
        raise TypeError(f"k_new: dtype {dtype} not in {tuple(_ROW_TYPES)}")
    T, stride = _check_new(k_new, v_new, start, cu_new, dtype, seqs, H, D)
    q_dtype = _check_rope(rope, positions, q, q_out, q_dtype, dtype, T, D)
    context, handle = _on(stream, (kv_pages, page_table, k_new, v_new, start, cu_new, rope, positions, q, q_out))
    with context:
        r, q_out = _make_rope(rope, positions, interleaved, q, q_out, q_dtype)
        _call("fathom_nibble_append", pages, kv_pages.data_ptr(), page_table.data_ptr(), _ROW_TYPES[dtype],
              k_new.data_ptr(), v_new.data_ptr(), T, stride[0], stride[1], start.data_ptr(),
              cu_new.data_ptr() if cu_new is not None else None, r, handle)
    return kv_pages, q_out


def fathom_nibble_read(pages: NibblePages, kv_pages, page_table, start, cu, total, dtype=torch.bfloat16, k_out=None,
                       v_out=None, stream=None):
    """Rows of a 4-bit cache: token i of sequence s's part (packed at cu[s] + i, `total` rows in all) is
    the one at position start[s] + i.  -> (k_out, v_out) [total][kv_heads][D] of dtype (bf16, fp16 or
    fp32; that of k_out if given); rows without a place in the cache are not written."""
    seqs, H, D = _check_nibble(pages, kv_pages, page_table)
    total = int(total)
    _fit32(total=total)
    if not _ok(start, torch.int32, (seqs,)):
        _check(start, "start", (torch.int32,), (seqs,))
    if not _ok(cu, torch.int32, (seqs + 1,)):
        _check(cu, "cu", (torch.int32,), (seqs + 1,))
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out: both or neither")
    if k_out is not None:
        dtype = k_out.dtype
        _check_strided(k_out, "k_out", tuple(_OUT_TYPES), (total, H, D))
        _check_strided(v_out, "v_out", (dtype,), (total, H, D))
        if any(a > 1 and x != y for a, x, y in zip((total, H), k_out.stride(), v_out.stride())):
            raise ValueError("v_out: strides differ from k_out's")
    elif dtype not in _OUT_TYPES:
        raise TypeError(f"dtype: {dtype} not in {tuple(_OUT_TYPES)}")
    elif total < 0:
        raise ValueError(f"total: {total} is negative")
    context, handle = _on(stream, (kv_pages, page_table, start, cu, k_out, v_out))
    with context:
        if k_out is None:
            k_out = torch.empty((total, H, D), dtype=dtype, device=kv_pages.device)
            v_out = torch.empty((total, H, D), dtype=dtype, device=kv_pages.device)
        _call("fathom_nibble_read", pages, kv_pages.data_ptr(), page_table.data_ptr(), start.data_ptr(), cu.data_ptr(),
              total, k_out.data_ptr(), v_out.data_ptr(), _OUT_TYPES[dtype], k_out.stride(0), k_out.stride(1), handle)
    return k_out, v_out


def nibble_workspace_size(pages: NibblePages, G: int) -> int:
    return int(lib().fathom_nibble_workspace_size(ctypes.byref(pages), int(G)))


def alloc_nibble_workspace(pages: NibblePages, G=4, device="cuda") -> torch.Tensor:
    """Workspace of fathom_nibble_attn.  One that is large enough for several calls of different sizes serves them in
    any order."""
    nbytes = nibble_workspace_size(pages, G)
    if nbytes == 0:
        raise FathomError("fathom_nibble_workspace_size", 1, lib().fathom_last_error().decode())
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def fathom_nibble_attn(pages: NibblePages, q, kv_pages, page_table, lens, workspace, out=None, lse=None, want_lse=False,
                       stream=None):
    """Decode attention over a 4-bit cache: q [units][G][D] fp32, lens [seqs] int32 -> out [units][G][D]
    fp32, or (out, lse [units][G] fp32) where lse is given or wanted."""
    seqs, H, D = _check_nibble(pages, kv_pages, page_table)
    if q is None or q.dim() != 3:
        raise ValueError("q: expected [units][G][D]")
    G = q.shape[1]
    shape = (seqs * H, G, D)
    if not _ok(q, torch.float32, shape):
        _check(q, "q", (torch.float32,), shape)
    if not _ok(lens, torch.int32, (seqs,)):
        _check(lens, "lens", (torch.int32,), (seqs,))
    if workspace is None or not (workspace.dtype is torch.uint8 and workspace.is_cuda and workspace.is_contiguous()):
        _check(workspace, "workspace", (torch.uint8,))
    if out is not None and not _ok(out, torch.float32, shape):
        _check(out, "out", (torch.float32,), shape)
    if lse is not None and not _ok(lse, torch.float32, shape[:2]):
        _check(lse, "lse", (torch.float32,), shape[:2])
    context, handle = _on(stream, (q, kv_pages, page_table, lens, workspace, out, lse))
    with context:
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=q.device)
        if lse is None and want_lse:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
        _call("fathom_nibble_attn", pages, G, q.data_ptr(), kv_pages.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
              out.data_ptr(), lse.data_ptr() if lse is not None else None, workspace.data_ptr(), workspace.numel(), handle)
    return out if lse is None else (out, lse)


def fathom_wait_status():
    """Synchronises the device; raises FathomError (status 4) if a bounded wait of the
    prompt attention ran out there since the last time it was asked."""
    _call("fathom_wait_status")


def fathom_debug_status(mode=0):
    """Debug build only: the first failed bounds check of the scan, gather and
    attention kernels, as three integers (site << 48 | index; 0: none).  mode 1
    also clears them; mode 2 plants a self-test record first."""
    out = (ctypes.c_uint64 * 3)()
    _call("fathom_debug_status", int(mode), ctypes.cast(out, ctypes.c_void_p))
    return [int(x) for x in out]
