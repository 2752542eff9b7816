"""e-means on MI355X: Python binding of libemeans.so.

Argument marshalling only: every step of the training and assignment runs in
the HIP kernels of ``libemeans.so``. PyTorch provides the device memory and the
stream; there is no CPU fallback. If the library is not built, every call
raises.

    import torch, mini_means_amd as mm
    x = torch.randn(100_000, 64, device="cuda")
    out = mm.train(x, k=1024)               # 5 passes, scaling-law recipe
    labels, dists = mm.assign(x, out.centroids)
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from dataclasses import dataclass
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libemeans.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "emeans.h")

MAX_PASSES = 64
F32, BF16, I8, F8, F16, U8 = 0, 1, 2, 3, 4, 5
LAWS = {"auto": 0, "throughput": 1, "quality": 2}
STATUS = {0: "OK", -1: "EINVAL", -2: "EDTYPE", -3: "ENOMEM", -4: "EHIP", -5: "ENOTDEVICE"}

c_i32, c_i64, c_dbl, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p


class Opts(ctypes.Structure):
    _fields_ = [
        ("dtype", c_i32), ("batch_law", c_i32), ("batch_size", c_i64), ("alpha0", c_dbl),
        ("unused_threshold", c_dbl), ("no_finalize", c_i32), ("profile", c_i32),
        ("stream", c_vp), ("trace_labels", c_vp), ("out_counts", c_vp), ("split_log", c_vp),
        ("split_log_cap", c_i64), ("max_steps", c_i64), ("bf16_search", c_i32),
        ("spherical", c_i32), ("lloyd", c_i32), ("slow_ema", c_dbl), ("slow_centroids", c_vp),
        ("search", c_i32), ("search_shift", c_vp), ("search_scale", c_dbl),
    ]


class Stats(ctypes.Structure):
    _fields_ = [
        ("batch_size", c_i64), ("total_steps", c_i64), ("n_splits", c_i64), ("n_logged", c_i64),
        ("dead_at_end", c_i64), ("alpha0", c_dbl), ("unused_threshold", c_dbl),
        ("law", c_i32), ("n_passes", c_i32),
        ("rows_per_pass", c_i64 * MAX_PASSES), ("steps_per_pass", c_i64 * MAX_PASSES),
        ("obj", c_dbl * MAX_PASSES), ("imbalance", c_dbl * MAX_PASSES),
        ("splits", c_i64 * MAX_PASSES),
        ("ms_total", c_dbl), ("ms_assign", c_dbl), ("ms_bucket", c_dbl), ("ms_group", c_dbl),
        ("ms_update", c_dbl),
        ("ms_revive", c_dbl), ("ms_sample", c_dbl), ("steps_run", c_i64),
        ("pass_ms", c_dbl * MAX_PASSES),
    ]


class EmeansError(RuntimeError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    """Load libemeans.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise EmeansError(f"{LIB_PATH} is missing: build it with "
                              "`python -m mini_means_amd.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        L.emeans_recipe.argtypes = [c_i64, c_i32, c_i32, c_dbl, ctypes.POINTER(Opts),
                                    ctypes.POINTER(Stats)]
        L.emeans_train.argtypes = [c_vp, c_i64, c_i32, c_i32, c_dbl, ctypes.c_uint64, c_vp, c_vp,
                                   ctypes.POINTER(Opts), ctypes.POINTER(Stats)]
        L.emeans_assign.argtypes = [c_vp, c_i64, c_i32, c_vp, c_i32, c_vp, c_vp,
                                    ctypes.POINTER(Opts)]
        L.emeans_assign_static.argtypes = L.emeans_assign.argtypes
        L.emeans_batch_rows.argtypes = [c_i64, ctypes.c_uint64, c_i32, c_i64, c_i64, c_vp, c_vp]
        L.emeans_begin.argtypes = [c_i64, c_i32, c_i32, c_dbl, ctypes.c_uint64, c_vp,
                                   ctypes.POINTER(Opts), ctypes.POINTER(c_vp)]
        L.emeans_accumulate.argtypes = [c_vp, c_vp, c_i64, c_vp]
        L.emeans_update.argtypes = [c_vp]
        L.emeans_end_epoch.argtypes = [c_vp]
        L.emeans_finalize.argtypes = [c_vp, c_vp, ctypes.POINTER(Stats)]
        L.emeans_closing_add.argtypes = [c_vp, c_vp, c_i64, c_vp, c_vp]
        L.emeans_free.argtypes = [c_vp]
        L.emeans_free.restype = None
        L.emeans_int8_calibrate.argtypes = [c_vp, c_i64, c_i32, c_vp, ctypes.POINTER(c_dbl), c_vp]
        L.emeans_int8_encode.argtypes = [c_vp, c_i64, c_i32, c_vp, c_dbl, c_vp, c_vp]
        L.emeans_int8_decode.argtypes = [c_vp, c_i64, c_i32, c_vp, c_dbl, c_vp, c_vp]
        for f in ("emeans_fp8_calibrate", "emeans_fp8_encode", "emeans_fp8_decode"):
            getattr(L, f).argtypes = getattr(L, f.replace("fp8", "int8")).argtypes
            getattr(L, f).restype = ctypes.c_int
        # lengths are 64 bits wide, as ctypes cuts what does not fit without a word
        L.emeans_block_encode.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_i32, c_vp, c_i64,
                                          c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp]
        L.emeans_block_matmul.argtypes = [c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64,
                                          c_i32, c_i64, c_i64, c_i64, c_vp, c_i32, c_i64, c_vp,
                                          c_vp]
        for f in ("emeans_block_matmul_work", "emeans_block_linear_work",
                  "emeans_block_train_saved"):
            getattr(L, f).argtypes = [c_i64, c_i64, c_i64]
            getattr(L, f).restype = c_i64
        L.emeans_block_linear.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_vp, c_i64, c_i32,
                                          c_i64, c_i64, c_i64, c_vp, c_i32, c_i64, c_vp, c_vp]
        L.emeans_block_train_saved_for.argtypes = [c_i64, c_i64, c_i64, c_i32]
        L.emeans_block_train_saved_for.restype = c_i64
        L.emeans_block_train_work.argtypes = [c_i64, c_i64, c_i64, c_i32]
        L.emeans_block_train_work.restype = c_i64
        L.emeans_block_train_forward.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i32, c_i64, c_i64,
                                                 c_i64, c_i64, c_i32, c_vp, c_i32, c_i64, c_vp,
                                                 c_vp, c_vp]
        L.emeans_block_train_gradient.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i64, c_i64, c_i64,
                                                  c_vp, c_i32, c_i64, c_vp, c_i32, c_i64, c_vp,
                                                  c_vp]
        L.emeans_cache_write.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp,
                                         c_i32, c_vp, c_vp, c_i64, c_i64, c_i32, c_vp]
        L.emeans_cache_read.argtypes = [c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_vp, c_i32,
                                        c_i64, c_vp, c_i32, c_i64, c_vp]
        L.emeans_cache_read_pages.argtypes = [c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_i32, c_vp,
                                              c_i64, c_i64, c_vp, c_i64, c_i64, c_vp, c_i32,
                                              c_i64, c_vp]
        rotate = [c_vp, c_i64, c_i64] * 2 + [c_i32, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_i32,
                                             c_vp, c_i32, c_vp, c_i64, c_dbl]
        L.emeans_norm_rotate.argtypes = rotate + [c_vp] * 3
        L.emeans_norm_rotate_gradient.argtypes = rotate + [c_vp, c_i64, c_i64] * 2 + [c_vp] * 6
        L.emeans_norm_rotate_work.argtypes = [c_i64, c_i64]
        attend = [c_vp, c_i64, c_i64] * 3 + [c_i32] + [c_i64] * 5 + [c_vp, c_vp, c_i64, c_i32, c_dbl]
        L.emeans_attend.argtypes = attend + [c_vp] * 4
        L.emeans_attend_gradient.argtypes = attend + [c_vp] * 4 + [c_i64, c_i64] + [c_vp] * 5
        L.emeans_attend_work.argtypes = [c_i64] * 6
        L.emeans_cache_attend_work.argtypes = [c_i64] * 6 + [c_i32]
        L.emeans_cache_attend.argtypes = [c_vp, c_i32, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_i64,
                                          c_i64, c_i64, c_i32, c_vp, c_i64, c_i64, c_vp, c_i64,
                                          c_i64, c_i64, c_i64, c_dbl, c_vp, c_vp, c_i64, c_vp,
                                          c_vp]
        L.emeans_cache_evict_work.argtypes = [c_i64, c_i64]
        L.emeans_cache_evict.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i32, c_i64, c_i64, c_vp, c_i64,
                                         c_i64, c_vp, c_i64, c_vp, c_i64, c_i64, c_i64, c_vp,
                                         c_vp, c_vp, c_vp, c_vp]
        for f in ("emeans_norm_rotate_work", "emeans_attend_work", "emeans_cache_attend_work",
                  "emeans_cache_evict_work"):
            getattr(L, f).restype = c_i64
        for f in ("emeans_norm_rotate", "emeans_norm_rotate_gradient", "emeans_attend",
                  "emeans_attend_gradient", "emeans_cache_attend", "emeans_cache_evict"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("emeans_block_encode", "emeans_block_matmul", "emeans_block_linear",
                  "emeans_block_train_forward", "emeans_block_train_gradient",
                  "emeans_cache_write", "emeans_cache_read", "emeans_cache_read_pages"):
            getattr(L, f).restype = ctypes.c_int
        L.emeans_last_error.restype = ctypes.c_char_p
        L.emeans_last_error.argtypes = []
        L.emeans_version.argtypes = []
        for f in ("emeans_recipe", "emeans_train", "emeans_assign", "emeans_assign_static",
                  "emeans_batch_rows",
                  "emeans_version", "emeans_begin", "emeans_accumulate", "emeans_update",
                  "emeans_end_epoch", "emeans_finalize", "emeans_closing_add",
                  "emeans_int8_calibrate",
                  "emeans_int8_encode", "emeans_int8_decode"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def declared_functions() -> list:
    """Function names the C header declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^\s*(?:int|int64_t|void|const char\*)\s+(emeans_\w+)\s*\(", text, flags=re.M)


def _check(rc: int) -> None:
    if rc != 0:
        msg = lib().emeans_last_error().decode(errors="replace")
        raise EmeansError(f"{STATUS.get(rc, rc)}: {msg}")


def _opts(dtype=F32, batch_law="auto", batch_size=0, alpha0=0.0, unused_threshold=None,
          finalize=True, profile=False, stream=None, lloyd=False) -> Opts:
    o = Opts()
    o.lloyd = 1 if lloyd else 0
    o.dtype = dtype
    o.batch_law = LAWS[batch_law] if isinstance(batch_law, str) else int(batch_law)
    o.batch_size = int(batch_size or 0)
    o.alpha0 = float(alpha0 or 0.0)
    # ABI: 0 = default, < 0 = off, > 0 = value; Python: None = default, 0 = off
    if unused_threshold is None:
        o.unused_threshold = 0.0
    elif unused_threshold <= 0:
        o.unused_threshold = -1.0
    else:
        o.unused_threshold = float(unused_threshold)
    o.no_finalize = 0 if finalize else 1
    o.profile = 1 if profile else 0
    o.stream = stream
    return o


SEARCH = {"bf16": BF16, "f16": F16, "fp16": F16, "f8": F8, "fp8": F8}


def _set_search(o: Opts, search, search_shift, search_scale, d: int):
    """On-the-fly search converter of fp32 data: search = 'bf16' | 'f16' |
    'f8' (None: none), search_shift = d float32 GPU tensor or None (centering
    for the casts, the FP8 converter's shift), search_scale (the FP8
    converter's power-of-two scale)."""
    if search is None:
        if search_shift is not None or search_scale is not None:
            raise EmeansError("EINVAL: search_shift / search_scale need search=")
        return
    if search not in SEARCH:
        raise EmeansError(f"EINVAL: search must be one of {sorted(SEARCH)} (got {search!r})")
    o.search = SEARCH[search]
    if search_shift is not None:
        _f32_device(search_shift, "search_shift")
        if search_shift.numel() != d:
            raise EmeansError(f"EINVAL: search_shift must have {d} values")
        o.search_shift = search_shift.data_ptr()
    o.search_scale = float(search_scale) if search_scale is not None else 0.0


def _stats_dict(s: Stats) -> dict:
    P = s.n_passes
    return dict(batch_size=s.batch_size, alpha0=s.alpha0, law=s.law, total_steps=s.total_steps,
                n_passes=P, epoch_rows=list(s.rows_per_pass[:P]),
                steps_per_pass=list(s.steps_per_pass[:P]), unused_threshold=s.unused_threshold,
                obj=list(s.obj[:P]), imbalance=list(s.imbalance[:P]), splits=list(s.splits[:P]),
                n_splits=s.n_splits, dead_at_end=s.dead_at_end, ms_total=s.ms_total,
                ms_assign=s.ms_assign, ms_bucket=s.ms_bucket, ms_group=s.ms_group,
                ms_update=s.ms_update,
                ms_revive=s.ms_revive, ms_sample=s.ms_sample, steps_run=s.steps_run,
                pass_ms=list(s.pass_ms[:P]))


def recipe(n: int, d: int, k: int, T: float = 5.0, **kw) -> dict:
    """Scaling-law recipe (host only): batch size, alpha0, passes and steps."""
    s = Stats()
    o = _opts(**kw)
    _check(lib().emeans_recipe(int(n), int(d), int(k), float(T), ctypes.byref(o), ctypes.byref(s)))
    return _stats_dict(s)


def _dtype_of(X) -> int:
    import torch
    if X.dtype == torch.float32:
        return F32
    if X.dtype == torch.bfloat16:
        return BF16
    if X.dtype == torch.int8:
        return I8
    if X.dtype == torch.float8_e4m3fn:
        return F8
    if X.dtype == torch.float16:
        return F16
    if X.dtype == torch.uint8:
        return U8
    raise EmeansError(f"EDTYPE: {X.dtype} not supported (float32, bfloat16, float16, int8, "
                      f"uint8 or float8_e4m3fn)")


def _stream_ptr(X, stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(X.device)
    return ctypes.c_void_p(s.cuda_stream)


def _require_device(X) -> None:
    if not getattr(X, "is_cuda", False):
        raise EmeansError("ENOTDEVICE: X must be a tensor on the GPU")
    if not X.is_contiguous():
        raise EmeansError("EINVAL: X must be contiguous")


@dataclass
class TrainOutput:
    centroids: object          # k x d float32 tensor
    labels: object             # n int32 tensor or None
    stats: dict
    trace: object = None       # int32 tensor of every step's labels, or None
    counts: object = None      # k float32 running counts at the end, or None
    split_log: Optional[list] = None
    slow_centroids: object = None  # k x d float32 slow-EMA centroids (slow_ema), or None


def train(X, k: int, T: float = 5.0, seed: int = 1234, *, batch_law="auto", batch_size: int = 0,
          alpha0: float = 0.0, unused_threshold=None, finalize: bool = True,
          capture_labels: bool = True, trace: bool = False, counts: bool = False,
          split_log_cap: int = 0, profile: bool = False, max_steps: int = 0,
          bf16_search: bool = False, spherical: bool = False, lloyd: bool = False,
          slow_ema: float = 0.0, search=None, search_shift=None, search_scale=None,
          stream=None) -> TrainOutput:
    """e-means training of X (n x d tensor on the GPU). lloyd: Lloyd
    iterations instead (T of them, every row each time, alpha = 1; clusters
    left without rows are split off donors after every iteration but the
    last, as Faiss's k-means does).
    slow_ema = kappa >= 1: also the centroids of a second, slower EMA over the
    last pass (rate alpha_t / kappa), for unseen data (out.slow_centroids).
    search = 'bf16' | 'f16' | 'f8' with search_shift / search_scale: fp32 rows
    converted batch by batch for the search (casts with optional centering,
    or the calibrated FP8 converter); results stay in data units."""
    import torch
    _require_device(X)
    n, d = X.shape
    dev = X.device
    with torch.cuda.device(dev):
        o = _opts(_dtype_of(X), batch_law, batch_size, alpha0, unused_threshold, finalize,
                  profile, _stream_ptr(X, stream), lloyd)
        rc = recipe(n, d, k, T, batch_law=batch_law, batch_size=batch_size, alpha0=alpha0,
                    unused_threshold=unused_threshold, lloyd=lloyd)
        C = torch.empty((k, d), dtype=torch.float32, device=dev)
        labels = torch.empty((n,), dtype=torch.int32, device=dev) if capture_labels else None
        tr = torch.empty((sum(rc["epoch_rows"]),), dtype=torch.int32, device=dev) if trace else None
        cn = torch.empty((k,), dtype=torch.float32, device=dev) if counts else None
        log = (ctypes.c_int32 * (3 * split_log_cap))() if split_log_cap > 0 else None
        if tr is not None:
            o.trace_labels = tr.data_ptr()
        if cn is not None:
            o.out_counts = cn.data_ptr()
        if log is not None:
            o.split_log = ctypes.cast(log, c_vp)
            o.split_log_cap = split_log_cap
        o.max_steps = int(max_steps)
        o.bf16_search = 1 if bf16_search else 0
        o.spherical = 1 if spherical else 0
        _set_search(o, search, search_shift, search_scale, d)
        SC = None
        if slow_ema:
            SC = torch.empty((k, d), dtype=torch.float32, device=dev)
            o.slow_ema = float(slow_ema)
            o.slow_centroids = SC.data_ptr()
        s = Stats()
        _check(lib().emeans_train(X.data_ptr(), n, d, int(k), float(T), int(seed) & (2**64 - 1),
                                  C.data_ptr(), labels.data_ptr() if labels is not None else None,
                                  ctypes.byref(o), ctypes.byref(s)))
        st = _stats_dict(s)
        splits = None
        if log is not None:
            m = min(s.n_logged, split_log_cap)
            splits = [(log[3 * i], log[3 * i + 1], log[3 * i + 2]) for i in range(m)]
        return TrainOutput(C, labels, st, tr, cn, splits, SC)


def assign(X, C, *, with_dists: bool = True, bf16_search: bool = False, spherical: bool = False,
           search=None, search_shift=None, search_scale=None, stream=None, no_alloc: bool = False,
           out=None):
    """Nearest centroid (int32 labels) and squared distance (float32) of each row.
    bf16_search: search fp32 rows in bf16 (rows and centroids rounded).
    search / search_shift / search_scale: the general converter (as train).
    spherical: the centroid of largest dot product, and that similarity.
    no_alloc: call emeans_assign_static (the library allocates nothing; its
    working memory is one fixed device array per GPU, shared by every call).
    out: (labels, dists or None) tensors to write into instead of new ones."""
    import torch
    _require_device(X)
    if not (getattr(C, "is_cuda", False) and C.dtype == torch.float32 and C.is_contiguous()):
        raise EmeansError("EINVAL: C must be a contiguous float32 tensor on the GPU")
    n, d = X.shape
    k = C.shape[0]
    if C.shape[1] != d:
        raise EmeansError("EINVAL: C and X differ in dimension")
    with torch.cuda.device(X.device):
        if out is not None:
            labels, dists = out
            if not (getattr(labels, "is_cuda", False) and labels.dtype == torch.int32
                    and labels.is_contiguous() and labels.numel() >= n):
                raise EmeansError("EINVAL: out labels must be a contiguous int32 GPU tensor of n")
            if dists is not None and not (getattr(dists, "is_cuda", False)
                                          and dists.dtype == torch.float32
                                          and dists.is_contiguous() and dists.numel() >= n):
                raise EmeansError("EINVAL: out dists must be a contiguous float32 GPU tensor of n")
        else:
            labels = torch.empty((n,), dtype=torch.int32, device=X.device)
            dists = torch.empty((n,), dtype=torch.float32, device=X.device) if with_dists else None
        o = _opts(_dtype_of(X), stream=_stream_ptr(X, stream))
        o.bf16_search = 1 if bf16_search else 0
        o.spherical = 1 if spherical else 0
        _set_search(o, search, search_shift, search_scale, d)
        fn = lib().emeans_assign_static if no_alloc else lib().emeans_assign
        if n:
            _check(fn(X.data_ptr(), n, d, C.data_ptr(), k, labels.data_ptr(),
                      dists.data_ptr() if dists is not None else None, ctypes.byref(o)))
    return labels, dists


def _f32_device(A, what: str):
    import torch
    if not (getattr(A, "is_cuda", False) and A.dtype == torch.float32 and A.is_contiguous()):
        raise EmeansError(f"EINVAL: {what} must be a contiguous float32 tensor on the GPU")


def _calibrate(sample, stream, fn):
    import torch
    _require_device(sample)
    _f32_device(sample, "sample")
    n, d = sample.shape
    shift = torch.empty((d,), dtype=torch.float32, device=sample.device)
    scale = c_dbl(0.0)
    with torch.cuda.device(sample.device):
        _check(getattr(lib(), fn)(sample.data_ptr(), n, d, shift.data_ptr(), ctypes.byref(scale),
                                  _stream_ptr(sample, stream)))
    return shift, scale.value


def _encode(X, shift, scale, stream, fn, dtype):
    import torch
    _require_device(X)
    _f32_device(X, "X")
    _f32_device(shift, "shift")
    n, d = X.shape
    if shift.numel() != d:
        raise EmeansError("EINVAL: shift must have d entries")
    codes = torch.empty((n, d), dtype=dtype, device=X.device)
    with torch.cuda.device(X.device):
        _check(getattr(lib(), fn)(X.data_ptr(), n, d, shift.data_ptr(), float(scale),
                                  codes.data_ptr(), _stream_ptr(X, stream)))
    return codes


def _decode(C, shift, scale, stream, fn):
    import torch
    _f32_device(C, "C")
    _f32_device(shift, "shift")
    k, d = C.shape
    if shift.numel() != d:
        raise EmeansError("EINVAL: shift must have d entries")
    out = torch.empty_like(C)
    with torch.cuda.device(C.device):
        _check(getattr(lib(), fn)(C.data_ptr(), k, d, shift.data_ptr(), float(scale),
                                  out.data_ptr(), _stream_ptr(C, stream)))
    return out


def int8_calibrate(sample, stream=None):
    """README "Data precision", INT8: per-dimension shift (d float32 tensor)
    and power-of-two scale (float) from sample rows (n x d float32 tensor)."""
    return _calibrate(sample, stream, "emeans_int8_calibrate")


def int8_encode(X, shift, scale: float, stream=None):
    """int8 codes of X (n x d float32 tensor): clamp(rint((X - shift) * scale), +-127)."""
    import torch
    return _encode(X, shift, scale, stream, "emeans_int8_encode", torch.int8)


def int8_decode(C, shift, scale: float, stream=None):
    """Code-space centroids (k x d float32 tensor) back to data space: C / scale + shift."""
    return _decode(C, shift, scale, stream, "emeans_int8_decode")


def fp8_calibrate(sample, stream=None):
    """README "Data precision", FP8: as int8_calibrate, for the +-448 range of E4M3."""
    return _calibrate(sample, stream, "emeans_fp8_calibrate")


def fp8_encode(X, shift, scale: float, stream=None):
    """FP8 E4M3 codes of X (a float8_e4m3fn tensor): the nearest E4M3 value of
    (X - shift) * scale, saturating at +-448."""
    import torch
    return _encode(X, shift, scale, stream, "emeans_fp8_encode", torch.float8_e4m3fn)


def fp8_decode(C, shift, scale: float, stream=None):
    """Code-space centroids back to data space: C / scale + shift."""
    return _decode(C, shift, scale, stream, "emeans_fp8_decode")


# ---- block codes: 8-bit codes with one power-of-two scale per block ----------
# These calls are short (a token's layer takes microseconds), so the checks read
# each attribute once.

BLOCK = 128  # values per scale of the matrix codes


class _Types:
    """torch and its types, looked up on first use."""
    torch = None


def _T():
    t = _Types
    if t.torch is None:
        import torch
        import torch.autograd.forward_ad as forward_ad
        t.numbers = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
        t.formats = {torch.float8_e4m3fn: F8, torch.int8: I8}
        t.codes = (torch.float8_e4m3fn,)
        t.bytes = (torch.float8_e8m0fnu, torch.uint8)
        t.stream = torch._C._cuda_getCurrentRawStream
        t.current = torch.cuda.current_device
        t.forward_ad = forward_ad
        t.dual = forward_ad.unpack_dual
        t.tracing = torch.jit.is_tracing
        t.torch = torch
    return t


def _number(dtype, what: str) -> int:
    code = _T().numbers.get(dtype)
    if code is None:
        raise EmeansError(f"EDTYPE: {what} {dtype} not supported (float32, bfloat16 or float16)")
    return code


def _device_of(X, what="X") -> int:
    if not getattr(X, "is_cuda", False):
        raise EmeansError(f"ENOTDEVICE: {what} must be a tensor on the GPU")
    return X.get_device()


def _elsewhere(device: int, stream):
    """The context a call has to enter: the given stream, so that new tensors
    are allocated where the library works, or the tensors' device; None where
    it is the current one already."""
    t = _T()
    if stream is not None:
        return t.torch.cuda.stream(stream)
    return t.torch.cuda.device(device) if device != t.current() else None


def _run(device: int, stream, call):
    """call(stream pointer) where the tensors live. A trace records torch's
    operations alone, so the library's would be missing from it."""
    if _T().tracing():
        raise EmeansError("EINVAL: calls of block codes cannot be traced (torch.jit.trace)")
    ctx = _elsewhere(device, stream)
    if ctx is None:
        return call(_T().stream(device))
    with ctx:
        return call(stream.cuda_stream if stream is not None else _T().stream(device))


def _matrix(A, device: int, what, dtypes, names):
    """A 2-D tensor on that device whose rows are runs of values: its rows,
    columns and row distance."""
    if not getattr(A, "is_cuda", False) or A.get_device() != device:
        raise EmeansError(f"ENOTDEVICE: {what} must be a tensor on the GPU of the others")
    if A.dtype not in dtypes:
        raise EmeansError(f"EDTYPE: {what} must be {names} (got {A.dtype})")
    shape = A.shape
    if len(shape) != 2:
        raise EmeansError(f"EINVAL: {what} must be 2-D with adjacent values in a row")
    n, d = shape
    ld, one = A.stride()
    if one != 1 and d > 1 and n:
        raise EmeansError(f"EINVAL: {what} must be 2-D with adjacent values in a row")
    return n, d, ld


def _room(n: int, d: int, unit: int, dtype, device):
    """n x d one-byte values with rows a multiple of `unit` bytes apart."""
    pitch = -(-d // unit) * unit
    room = _T().torch.empty((n, pitch), dtype=dtype, device=device)
    return room if pitch == d else room[:, :d]


def block_encode(X, *, tiles: bool = False, rows: bool = True, cols: bool = False, stream=None):
    """E4M3 codes of X (n x d float32, bfloat16 or float16 tensor on the GPU,
    rows any distance apart) with one power-of-two scale for each 128 values
    (float8_e8m0fnu): the smallest s with max |x| <= 448 s, codes the nearest
    E4M3 values of x / s.

    Returns (codes n x d, scales n x ceil(d/128)), blocks along the rows; with
    cols=True (codes, scales, codes_t, scales_t), where codes_t (d x n) and
    scales_t (d x ceil(n/128)) are the transpose with blocks along its rows, made
    from the same read of X (rows=False: the first two are None). tiles=True:
    a block is a 128 x 128 tile, scales ceil(n/128) x ceil(d/128), and both
    orders hold the same codes (the form for weights). Rows of codes start at
    multiples of 16 bytes: for other d the tensors are views of wider ones."""
    dev = _device_of(X)
    dt = _number(X.dtype, "X")
    n, d, ldx = _matrix(X, dev, "X", (X.dtype,), "")
    if not rows and not cols:
        raise EmeansError("EINVAL: block_encode makes rows, cols or both")
    if ldx < d and n > 1:
        raise EmeansError("EINVAL: the rows of X overlap")
    nb, db = -(-n // BLOCK), -(-d // BLOCK)

    def call(st):
        f8, e8 = _T().codes[0], _T().bytes[0]
        out = [None] * 4
        if rows:
            out[0] = _room(n, d, 16, f8, X.device)
            out[1] = _room(nb if tiles else n, db, 4, e8, X.device)
        if cols:
            out[2] = _room(d, n, 16, f8, X.device)
            out[3] = _room(db if tiles else d, nb, 4, e8, X.device)
        if n and d:
            args = [v for t in out for v in ((None, 0) if t is None else (t.data_ptr(), t.stride(0)))]
            _check(lib().emeans_block_encode(X.data_ptr(), dt, n, d, ldx, 1 if tiles else 0, *args,
                                             st))
        return tuple(out) if cols else (out[0], out[1])

    return _run(dev, stream, call)


def _product_side(dev, codes, scales, what):
    """Rows, columns and row distances of one side of the product, and whether
    its scales stand per tile."""
    t = _T()
    n, k, ld = _matrix(codes, dev, what, t.codes, "float8_e4m3fn codes")
    sn, sk, lds = _matrix(scales, dev, "its scales", t.bytes, "float8_e8m0fnu or uint8 scales")
    if sk != -(-k // BLOCK) or (sn != n and sn != -(-n // BLOCK)):
        raise EmeansError(f"EINVAL: scales of {what} must be {n} x {-(-k // BLOCK)} (rows) or "
                          f"{-(-n // BLOCK)} x {-(-k // BLOCK)} (tiles), got {sn} x {sk}")
    return n, k, ld, lds, sn != n


def _product_out(m, n, out, out_dtype, device):
    if out is None:
        return _T().torch.empty((m, n), dtype=out_dtype, device=device)
    if not (getattr(out, "is_cuda", False) and out.device == device and out.dtype == out_dtype
            and out.shape == (m, n) and (out.stride(1) == 1 or n <= 1)):
        raise EmeansError(f"EINVAL: out must be an {m} x {n} {out_dtype} GPU tensor with adjacent "
                          "values in a row")
    return out


def _ptr(t):
    """Address of a tensor; None for none."""
    return None if t is None else t.data_ptr()


def _work(need: int, device):
    """Working memory of one call, allocated where the call runs; None for none."""
    return _T().torch.empty((need,), dtype=_T().torch.uint8, device=device) if need else None


def block_matmul(a, a_scales, b, b_scales, *, out_dtype=None, out=None, stream=None):
    """a b^T (m x n) of block codes: a m x k and b n x k float8_e4m3fn tensors
    with scales per row and 128 values (as block_encode makes them); b_scales
    may instead stand per 128 x 128 tile. out: a tensor to write into.

    Rounded once to out_dtype: float32 (sums in fp32), bfloat16 (the default) or
    float16. Results of 16 bits are sums of the FP8 matrix unit, which keeps 13
    bits below the largest of each eight consecutive products: off by less than
    2^-10 of the sum of |a b| whatever the data, by 1.5e-5 of the result's norm on
    normal values, up to 7e-5 on activations with a few large columns (the
    rounding to bfloat16 1.7e-3, float16 2.1e-4). Ask for float32 where the terms
    cancel. The same call gives the same bits; a row's last bits may change with
    the number of rows beside it."""
    out_dtype = out_dtype or (out.dtype if out is not None else _T().torch.bfloat16)
    ot = _number(out_dtype, "out_dtype")
    dev = _device_of(a, "a")
    m, k, lda, ldas, a_tiles = _product_side(dev, a, a_scales, "a")
    n, kb, ldb, ldbs, b_tiles = _product_side(dev, b, b_scales, "b")
    if kb != k:
        raise EmeansError(f"EINVAL: a has {k} columns, b has {kb}")
    if a_tiles:
        raise EmeansError("EINVAL: a_scales must stand per row (tiles are for b)")

    def call(st):
        y = _product_out(m, n, out, out_dtype, a.device)
        if m and n:
            L = lib()
            work = _work(L.emeans_block_matmul_work(m, n, k), a.device)
            _check(L.emeans_block_matmul(a.data_ptr(), lda, a_scales.data_ptr(), ldas,
                                         b.data_ptr(), ldb, b_scales.data_ptr(), ldbs,
                                         1 if b_tiles else 0, m, n, k, y.data_ptr(), ot,
                                         y.stride(0), _ptr(work), st))
        return y

    return _run(dev, stream, call)


def _linear_codes(x, w, w_scales, out_dtype):
    """x (m x k numbers) times the transpose of codes: one library call."""
    dev = x.get_device()
    dt = _number(x.dtype, "X")
    ot = _number(out_dtype, "out_dtype")
    m, k, ldx = _matrix(x, dev, "X", (x.dtype,), "")
    n, kw, ldb, ldbs, tiles = _product_side(dev, w, w_scales, "w")
    if kw != k:
        raise EmeansError(f"EINVAL: X has {k} columns, w has {kw}")

    def call(st):
        y = _T().torch.empty((m, n), dtype=out_dtype, device=x.device)
        if m and n:
            L = lib()
            work = _work(L.emeans_block_linear_work(m, n, k), x.device)
            _check(L.emeans_block_linear(x.data_ptr(), dt, ldx, w.data_ptr(), ldb,
                                         w_scales.data_ptr(), ldbs, 1 if tiles else 0, m, n, k,
                                         y.data_ptr(), ot, n, _ptr(work), st))
        return y

    return _run(dev, None, call)


def _tiles_room(n: int, d: int):
    """One room for the codes of an n x d matrix with a scale per tile: the codes'
    row distance, where the scales start, their row distance, bytes in all."""
    ld, lds = -(-d // 16) * 16, -(-d // (4 * BLOCK)) * 4
    return ld, n * ld, lds, -(-(n * ld + -(-n // BLOCK) * lds) // 16) * 16


def _rows(t):
    """t as a matrix whose rows are runs that do not overlap (a copy if it is
    not one: an expanded gradient, say)."""
    n, d = t.shape
    ld, one = t.stride()
    return t if (one == 1 or d <= 1) and (ld >= d or n <= 1) else t.contiguous()


_linear_function = None


def _linear_fn():
    global _linear_function
    if _linear_function is None:
        torch = _T().torch

        class BlockLinear(torch.autograd.Function):
            """y = Q(x) Q(w)^T; the rounding passes gradients straight through."""

            @staticmethod
            def forward(ctx, x, w, out_dtype):
                dev = x.get_device()
                dt, wt = _number(x.dtype, "X"), _number(w.dtype, "w")
                ot = _number(out_dtype, "out_dtype")
                m, k, ldx = _matrix(x, dev, "X", (x.dtype,), "")
                n, _, ldw = _matrix(w, dev, "w", (w.dtype,), "")
                if n < 1 or k < 1:
                    raise EmeansError("EINVAL: w must have rows and columns")
                need = sum(b for b, g in zip((1, 2), ctx.needs_input_grad) if g)
                L = lib()

                def call(st):
                    y = torch.empty((m, n), dtype=out_dtype, device=x.device)
                    saved = _work(L.emeans_block_train_saved_for(m, n, k, need), x.device)
                    work = _work(L.emeans_block_train_work(m, n, k, 0), x.device)
                    if m:
                        _check(L.emeans_block_train_forward(
                            x.data_ptr(), dt, ldx, w.data_ptr(), wt, ldw, m, n, k, need,
                            y.data_ptr(), ot, n, _ptr(saved), _ptr(work), st))
                    return y, saved

                y, saved = _run(dev, None, call)
                ctx.save_for_backward(saved)
                ctx.args = m, n, k, x.dtype, dt, w.dtype, wt
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                saved, = ctx.saved_tensors
                m, n, k, x_type, dt, w_type, wt = ctx.args
                need_x, need_w = ctx.needs_input_grad[:2]
                L = lib()

                def call(st):
                    g = _rows(dy)
                    dx = torch.empty((m, k), dtype=x_type, device=g.device) if need_x else None
                    dw = torch.empty((n, k), dtype=w_type, device=g.device) if need_w else None
                    work = _work(L.emeans_block_train_work(m, n, k, 1), g.device)
                    if m or need_w:
                        _check(L.emeans_block_train_gradient(
                            g.data_ptr(), _number(g.dtype, "the gradient"), g.stride(0),
                            saved.data_ptr() if m else None, m, n, k,
                            dx.data_ptr() if need_x else None, dt, k,
                            dw.data_ptr() if need_w else None, wt, k,
                            work.data_ptr() if m else None, st))
                    return dx, dw

                return *_run(dy.get_device(), None, call), None

        class BlockLinearFrozen(torch.autograd.Function):
            """The same with w as codes in both orders: a gradient of x alone."""

            @staticmethod
            def forward(ctx, x, frozen, out_dtype):
                w, s, wc, wcs = frozen
                ctx.save_for_backward(wc, wcs)
                ctx.x_type = x.dtype
                return _linear_codes(x, w, s, out_dtype)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                wc, wcs = ctx.saved_tensors
                return _linear_codes(_rows(dy), wc, wcs, ctx.x_type), None, None

        class BlockLinearX(torch.autograd.Function):
            """The same with a gradient of x alone: w's transposed codes are kept."""

            @staticmethod
            def forward(ctx, x, w, out_dtype):
                dev = x.get_device()
                dt, wt = _number(x.dtype, "X"), _number(w.dtype, "w")
                ot = _number(out_dtype, "out_dtype")
                m, k, ldx = _matrix(x, dev, "X", (x.dtype,), "")
                n, _, ldw = _matrix(w, dev, "w", (w.dtype,), "")
                if n < 1 or k < 1:
                    raise EmeansError("EINVAL: w must have rows and columns")
                L = lib()
                ld, scales, lds, size = _tiles_room(n, k)
                ldt, scales_t, ldst, size_t = _tiles_room(k, n)

                def call(st):
                    y = torch.empty((m, n), dtype=out_dtype, device=x.device)
                    kept = _work(size_t, x.device)
                    if m:
                        work = _work(size + L.emeans_block_linear_work(m, n, k), x.device)
                        at, at_t = work.data_ptr(), kept.data_ptr()
                        _check(L.emeans_block_encode(w.data_ptr(), wt, n, k, ldw, 1, at, ld,
                                                     at + scales, lds, at_t, ldt, at_t + scales_t,
                                                     ldst, st))
                        _check(L.emeans_block_linear(x.data_ptr(), dt, ldx, at, ld, at + scales,
                                                     lds, 1, m, n, k, y.data_ptr(), ot, n,
                                                     at + size, st))
                    return y, kept

                y, kept = _run(dev, None, call)
                ctx.save_for_backward(kept)
                ctx.args = m, n, k, x.dtype, dt
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                kept, = ctx.saved_tensors
                m, n, k, x_type, dt = ctx.args
                ldt, scales_t, ldst, _ = _tiles_room(k, n)
                L = lib()

                def call(st):
                    g = _rows(dy)
                    dx = torch.empty((m, k), dtype=x_type, device=g.device)
                    if m:
                        work = _work(L.emeans_block_linear_work(m, k, n), g.device)
                        at = kept.data_ptr()
                        _check(L.emeans_block_linear(g.data_ptr(), _number(g.dtype, "the gradient"),
                                                     g.stride(0), at, ldt, at + scales_t, ldst, 1,
                                                     m, k, n, dx.data_ptr(), dt, k, _ptr(work), st))
                    return dx

                return _run(dy.get_device(), None, call), None, None

        _linear_function = BlockLinear, BlockLinearFrozen, BlockLinearX
    return _linear_function


def block_linear(X, w, *, out_dtype=None, stream=None):
    """y = X w^T (X (..., k), w n x k) with both sides as block codes: X encoded
    along its rows, w in 128 x 128 tiles; y in out_dtype (X's by default). Sums as
    in block_matmul: y, dX and dw of 16 bits are the FP8 unit's, float32 ones fp32.

    w a float32, bfloat16 or float16 tensor: encoded in the call; gradients of
    X and w pass straight through the rounding, dX = Q(dY) Q(w) and dw =
    Qt(dY) Qt(X)^T (Qt: the transpose, blocks along the rows of X), with the codes
    of X (if w has a gradient) and of w (if X has one) kept for the backward pass
    instead of the numbers.
    w a tuple (codes, scales), as block_encode(w, tiles=True) gives: serving,
    where a few rows of X are encoded inside the product's launch. With the
    tuple of four of block_encode(w, tiles=True, cols=True), X has a gradient
    and the frozen w none. Gradients are those of the backward pass, once: tangents
    of the forward mode are refused.

    On `stream` (the current one by default) everything runs, copies of inputs
    whose values are not adjacent too; the backward pass as well, ordered behind
    its gradient by autograd."""
    _device_of(X)
    if stream is not None:
        with _T().torch.cuda.stream(stream):
            return block_linear(X, w, out_dtype=out_dtype)
    dual, coded = _T().dual, isinstance(w, (tuple, list))
    if dual(X).tangent is not None or not coded and dual(w).tangent is not None:
        raise EmeansError("EINVAL: block_linear has no forward-mode derivative (X or w has a tangent)")
    out_dtype = out_dtype or X.dtype
    flat = X.dim() == 2
    if X.dim() == 0:
        raise EmeansError("EINVAL: X must have rows of k values")
    x = X if flat else X.reshape(math.prod(X.shape[:-1]), X.shape[-1])
    grad = _T().torch.is_grad_enabled()
    if coded:
        if len(w) not in (2, 4):
            raise EmeansError("EINVAL: w must be a tensor, (codes, scales) or the four of "
                              "block_encode(w, tiles=True, cols=True)")
        if grad and X.requires_grad:
            if len(w) != 4:
                raise EmeansError("EINVAL: the gradient of X needs the transposed codes of w: pass "
                                  "the four of block_encode(w, tiles=True, cols=True)")
            y = _linear_fn()[1].apply(_rows(x), tuple(w), out_dtype)
        else:
            y = _linear_codes(_rows(x), w[0], w[1], out_dtype)
    else:
        if w.dim() != 2 or w.shape[1] != x.shape[1]:
            raise EmeansError(f"EINVAL: w must be n x {x.shape[1]}")
        if grad and w.requires_grad:
            y = _linear_fn()[0].apply(_rows(x), _rows(w), out_dtype)
        elif grad and X.requires_grad:
            y = _linear_fn()[2].apply(_rows(x), _rows(w), out_dtype)
        else:
            y = _linear_codes(_rows(x), *block_encode(_rows(w), tiles=True), out_dtype)
    return y if flat else y.view(*X.shape[:-1], y.shape[1])


def _check_block(block) -> None:
    if not 16 <= block <= 256 or block % 16:
        raise EmeansError(f"EINVAL: block must be a multiple of 16 in [16, 256] (got {block})")


def cache_new(rows, d: int, *, block: int = BLOCK, dtype=None, device="cuda"):
    """An empty store of codes: (codes, scales) of shape rows + (d,) and rows +
    (ceil(d / block),), rows a number or a shape such as (pages, rows per
    page). dtype float8_e4m3fn (default) or int8. Its rows read as zeros."""
    torch = _T().torch
    shape = tuple(rows) if hasattr(rows, "__iter__") else (rows,)
    dtype = dtype or torch.float8_e4m3fn
    if dtype not in _T().formats:
        raise EmeansError(f"EDTYPE: {dtype} not supported (float8_e4m3fn or int8)")
    _check_block(block)
    codes = torch.zeros((*shape, d), dtype=torch.uint8, device=device).view(dtype)
    scales = torch.full((*shape, -(-d // block)), 127, dtype=torch.uint8, device=device)
    return codes, scales.view(torch.float8_e8m0fnu)


def _store(dev, codes, scales, block):
    """Format, rows and row length of a store."""
    t = _T()
    fmt = t.formats.get(codes.dtype)
    if fmt is None:
        raise EmeansError(f"EDTYPE: codes must be float8_e4m3fn or int8 (got {codes.dtype})")
    if scales.dtype not in t.bytes:
        raise EmeansError(f"EDTYPE: scales must be float8_e8m0fnu or uint8 (got {scales.dtype})")
    if not codes.is_cuda or not scales.is_cuda or codes.get_device() != dev \
            or scales.get_device() != dev:
        raise EmeansError("ENOTDEVICE: codes and scales must be tensors on the GPU of the others")
    shape, sshape = codes.shape, scales.shape
    if len(shape) < 2 or not codes.is_contiguous() or not scales.is_contiguous():
        raise EmeansError("EINVAL: codes and scales must be contiguous, rows last but one")
    d = shape[-1]
    _check_block(block)
    if shape[:-1] != sshape[:-1] or sshape[-1] != -(-d // block):
        raise EmeansError(f"EINVAL: scales must be {tuple(shape[:-1])} x ceil({d} / {block}), got "
                          f"{tuple(sshape)}")
    return fmt, codes.numel() // d if d else 0, d


def _slots(dev, slots, n=None):
    if not getattr(slots, "is_cuda", False) or slots.get_device() != dev:
        raise EmeansError("ENOTDEVICE: slots must be a tensor on the GPU of the others")
    torch = _T().torch
    dtype = slots.dtype
    if dtype is not torch.int64 and dtype is not torch.int32:
        raise EmeansError(f"EDTYPE: slots must be int32 or int64 (got {dtype})")
    if slots.dim() != 1 or not slots.is_contiguous() or (n is not None and slots.shape[0] != n):
        raise EmeansError("EINVAL: slots must be one contiguous number per row")
    return 8 if dtype is torch.int64 else 4


def cache_write(X, slots, codes, scales, *, block: int = BLOCK, stream=None) -> None:
    """Encode the rows of X (n x d, or n x heads x width with any distance
    between rows and between heads; float32, bfloat16 or float16) into the rows
    of a store (cache_new) that slots (n int32 or int64, distinct) names, with
    one scale for each `block` values of a row. The store may have any shape
    rows x d, pages x page rows x d, ...: a slot counts its rows in order.
    Negative slots and slots past its end are skipped."""
    dev = _device_of(X)
    dt = _number(X.dtype, "X")
    fmt, rows, d = _store(dev, codes, scales, block)
    shape, stride = X.shape, X.stride()
    if len(shape) not in (2, 3) or (stride[-1] != 1 and shape[-1] > 1):
        raise EmeansError("EINVAL: X must be n x d or n x heads x width with adjacent values")
    n, heads, width = (shape[0], 1, shape[1]) if len(shape) == 2 else shape
    if heads * width != d:
        raise EmeansError(f"EINVAL: X has rows of {heads * width} values, the store of {d}")
    size = _slots(dev, slots, n)
    if n and rows:
        _run(dev, stream, lambda st: _check(lib().emeans_cache_write(
            X.data_ptr(), dt, n, heads, width, stride[0], stride[1] if len(shape) == 3 else width,
            slots.data_ptr(), size, codes.data_ptr(), scales.data_ptr(), rows, block, fmt, st)))


def cache_read(codes, scales, slots, *, block: int = BLOCK, out_dtype=None, out=None, stream=None):
    """Rows slots (int32 or int64) of a store as numbers (len(slots) x d,
    out_dtype: bfloat16 by default, float32 or float16). A slot outside the
    store reads as zeros. out: a tensor to write into."""
    out_dtype = out_dtype or (out.dtype if out is not None else _T().torch.bfloat16)
    ot = _number(out_dtype, "out_dtype")
    dev = _device_of(codes, "codes")
    fmt, rows, d = _store(dev, codes, scales, block)
    size = _slots(dev, slots)
    n = slots.shape[0]

    def call(st):
        y = _product_out(n, d, out, out_dtype, codes.device)
        if n:
            _check(lib().emeans_cache_read(codes.data_ptr(), scales.data_ptr(), rows, d, block,
                                           fmt, slots.data_ptr(), size, n, y.data_ptr(), ot,
                                           y.stride(0), st))
        return y

    return _run(dev, stream, call)


def cache_read_pages(codes, scales, table, starts, total: int, *, block: int = BLOCK,
                     out_dtype=None, out=None, stream=None):
    """Ragged sequences of a paged store (codes pages x page rows x d) packed
    into total x d numbers: sequence s is rows starts[s] .. starts[s + 1] of the
    result (starts: seqs + 1 int32), its row p in page table[s, p // page rows]
    (table: seqs x pages of the longest, int32). Rows of the result outside
    every sequence, and rows whose page is negative or past the end, are zeros.
    total is the host's number: nothing is read back."""
    torch = _T().torch
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    ot = _number(out_dtype, "out_dtype")
    dev = _device_of(codes, "codes")
    fmt, _, d = _store(dev, codes, scales, block)
    if codes.dim() != 3:
        raise EmeansError("EINVAL: codes must be pages x page rows x d")
    seqs, table_pages, ldt = _matrix(table, dev, "table", (torch.int32,), "int32")
    if not getattr(starts, "is_cuda", False) or starts.get_device() != dev:
        raise EmeansError("ENOTDEVICE: starts must be a tensor on the GPU of the others")
    if starts.dtype is not torch.int32 or not starts.is_contiguous() or starts.shape != (seqs + 1,):
        raise EmeansError(f"EINVAL: starts must be {seqs + 1} contiguous int32")
    total = int(total)
    if total < 0:
        raise EmeansError(f"EINVAL: total out of range ({total})")

    def call(st):
        y = _product_out(total, d, out, out_dtype, codes.device)
        if total:
            _check(lib().emeans_cache_read_pages(
                codes.data_ptr(), scales.data_ptr(), codes.shape[0], codes.shape[1], d, block,
                fmt, table.data_ptr(), ldt, table_pages, starts.data_ptr(), seqs, total,
                y.data_ptr(), ot, y.stride(0), st))
        return y

    return _run(dev, stream, call)


# ---- attention around the store ----------------------------------------------


def _heads(A, device: int, what, dtype=None):
    """A tensor n x heads x width on that device whose heads are runs of values:
    its sizes and the distances of rows and heads."""
    if not getattr(A, "is_cuda", False) or A.get_device() != device:
        raise EmeansError(f"ENOTDEVICE: {what} must be a tensor on the GPU of the others")
    if dtype is not None and A.dtype != dtype:
        raise EmeansError(f"EDTYPE: {what} must be {dtype} (got {A.dtype})")
    shape = A.shape
    if len(shape) != 3 or (A.stride(2) != 1 and shape[2] > 1 and A.numel()):
        raise EmeansError(f"EINVAL: {what} must be rows x heads x width with adjacent values")
    return (*shape, A.stride(0), A.stride(1))


def _vector(A, device: int, what, n, dtypes, names):
    """A contiguous 1-D tensor of n values (any number where n is None)."""
    if not getattr(A, "is_cuda", False) or A.get_device() != device:
        raise EmeansError(f"ENOTDEVICE: {what} must be a tensor on the GPU of the others")
    if A.dtype not in dtypes:
        raise EmeansError(f"EDTYPE: {what} must be {names} (got {A.dtype})")
    if A.dim() != 1 or not A.is_contiguous() or (n is not None and A.shape[0] != n):
        raise EmeansError(f"EINVAL: {what} must be {'contiguous' if n is None else n} "
                          f"{names} values in a row")
    return A.shape[0]


def _no_tangent(name, *tensors) -> None:
    t = _T()
    if t.forward_ad._current_level < 0:
        return  # no level of the forward mode is entered, so no tensor has a tangent
    if any(t.dual(x).tangent is not None for x in tensors):
        raise EmeansError(f"EINVAL: {name} has no forward-mode derivative (an input has a tangent)")


def _no_gradient(name, x) -> None:
    """Refuse an input that asks for a gradient that the call does not have."""
    t = _T()
    if getattr(x, "requires_grad", False) and t.torch.is_grad_enabled():
        raise EmeansError(f"EINVAL: {name} has no gradient (detach the input that asks for one)")
    if t.forward_ad._current_level >= 0:
        _no_tangent(name, x)


def _adjacent(t):
    """t with adjacent values in a row (a copy if it has not)."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def rotary_freqs(turned: int, base: float = 10000.0, device="cuda"):
    """Radians per position of the turned / 2 pairs of a head, base^(-2 i / turned)
    (float64), as norm_rotate takes them. turned: a multiple of 8."""
    torch = _T().torch
    if turned < 0 or turned % 8 or not base > 0:
        raise EmeansError(f"EINVAL: turned must be a multiple of 8 and base positive (got {turned}, "
                          f"{base})")
    i = torch.arange(turned // 2, dtype=torch.float64, device=device)
    return torch.exp2(i * (-2.0 * math.log2(base) / max(turned, 1)))


def _rotate_args(q, k, q_weight, k_weight, positions, freqs, eps):
    """The arguments that both passes of norm_rotate share, and the sizes."""
    dev, gt, half = _rotate_checks(q, k, q_weight, k_weight, positions, freqs)
    return dev, _rotate_list(q, k, q_weight, k_weight, positions, freqs, gt, half, eps)


def _rotate_list(q, k, q_weight, k_weight, positions, freqs, gt, half, eps):
    n, hq, w = q.shape
    qs, ks = q.stride(), k.stride()
    t = _T()
    return (q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], t.numbers[q.dtype], n, hq,
            k.shape[1], w, q_weight.data_ptr(), k_weight.data_ptr(), gt, positions.data_ptr(),
            8 if positions.dtype is t.torch.int64 else 4, freqs.data_ptr(), half, eps)


def _rotate_checks(q, k, q_weight, k_weight, positions, freqs):
    t = _T()
    dev = _device_of(q, "q")
    _number(q.dtype, "q")
    n, _, w, _, _ = _heads(q, dev, "q")
    nk, _, wk, _, _ = _heads(k, dev, "k", q.dtype)
    if nk != n or wk != w:
        raise EmeansError(f"EINVAL: k must be {n} x heads x {w} (got {tuple(k.shape)})")
    gt = _number(q_weight.dtype, "q_weight")
    names = str(q_weight.dtype)
    _vector(q_weight, dev, "q_weight", w, (q_weight.dtype,), names)
    _vector(k_weight, dev, "k_weight", w, (q_weight.dtype,), names)
    _vector(positions, dev, "positions", n, (t.torch.int32, t.torch.int64), "int32 or int64")
    return dev, gt, _vector(freqs, dev, "freqs", None, (t.torch.float64,), "float64")


def _norm_rotate(q, k, q_weight, k_weight, positions, freqs, eps):
    dev, args = _rotate_args(q, k, q_weight, k_weight, positions, freqs, eps)

    def call(st):
        empty, device = _T().torch.empty, q.device
        qo = empty(q.shape, dtype=q.dtype, device=device)
        ko = empty(k.shape, dtype=q.dtype, device=device)
        _check(lib().emeans_norm_rotate(*args, qo.data_ptr(), ko.data_ptr(), st))
        return qo, ko

    return _run(dev, None, call)


_rotate_function = None


def _rotate_fn():
    global _rotate_function
    if _rotate_function is None:
        torch = _T().torch

        class NormRotate(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_weight, k_weight, positions, freqs, eps):
                ctx.save_for_backward(q, k, q_weight, k_weight, positions, freqs)
                ctx.eps = eps
                return _norm_rotate(q, k, q_weight, k_weight, positions, freqs, eps)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dqo, dko):
                q, k, gq, gk, positions, freqs = ctx.saved_tensors
                L, dtype, device = lib(), q.dtype, q.device
                args = _rotate_list(q, k, gq, gk, positions, freqs, _T().numbers[gq.dtype],
                                    freqs.shape[0], ctx.eps)

                def call(st):
                    a, b = _adjacent(dqo), _adjacent(dko)
                    dq, dk = (torch.empty(x.shape, dtype=dtype, device=device) for x in (q, k))
                    dgq, dgk = (torch.empty(gq.shape, dtype=gq.dtype, device=device) for _ in "qk")
                    work = _work(L.emeans_norm_rotate_work(q.shape[0], q.shape[2]), device)
                    sa, sb = a.stride(), b.stride()
                    _check(L.emeans_norm_rotate_gradient(
                        *args, a.data_ptr(), sa[0], sa[1], b.data_ptr(), sb[0], sb[1],
                        dq.data_ptr(), dk.data_ptr(), dgq.data_ptr(), dgk.data_ptr(), _ptr(work),
                        st))
                    return dq, dk, dgq, dgk

                return *_run(q.get_device(), None, call), None, None, None

        _rotate_function = NormRotate
    return _rotate_function


def norm_rotate(q, k, q_weight, k_weight, positions, freqs, *, eps: float = 1e-6, stream=None):
    """Queries (n x hq x width) and keys (n x hk x width; float32, bfloat16 or
    float16, rows and heads any distance apart) normed per head and turned by their
    positions in one pass: y = x / sqrt(mean x^2 + eps) * weight, then the pairs
    (c, c + half) turned by positions[t] * freqs[c], half = len(freqs); values from
    2 half on are only normed. Returns the two results (contiguous, one rounding).

    width is a multiple of 8 up to 256, half a multiple of 4. The weights (width
    values) are both of one number type, positions (n) int32 or int64, freqs float64
    (rotary_freqs): angles are exact products in 64 bits, so far positions turn as
    exactly as near ones. q, k and the weights have gradients (once: tangents of the
    forward mode are refused, and freqs that ask for a gradient); the weights' are sums
    in one order."""
    _device_of(q, "q")
    if stream is not None:
        with _T().torch.cuda.stream(stream):
            return norm_rotate(q, k, q_weight, k_weight, positions, freqs, eps=eps)
    _no_tangent("norm_rotate", q, k, q_weight, k_weight)
    _no_gradient("norm_rotate by freqs", freqs)
    if _T().torch.is_grad_enabled() and (q.requires_grad or k.requires_grad
                                         or q_weight.requires_grad or k_weight.requires_grad):
        return _rotate_fn().apply(q, k, q_weight, k_weight, positions, freqs, eps)
    return _norm_rotate(q, k, q_weight, k_weight, positions, freqs, eps)


def _aligned(t):
    """t with heads of adjacent values at multiples of 16 bytes (a copy if they are not)."""
    a, b, c = t.stride()
    if (c == 1 or t.shape[2] <= 1) and a % 8 == 0 and b % 8 == 0 and t.data_ptr() % 16 == 0 \
            and a < 1 << 24:
        return t
    # not contiguous(): that returns t itself where what is oddly apart is one row or head
    return t.clone(memory_format=_T().torch.contiguous_format)


def _attend_list(q, k, v, starts, k_starts, causal, scale):
    """The arguments that both passes of attend share."""
    n, hq, w = q.shape
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    return (q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
            _T().numbers[q.dtype], n, k.shape[0], hq, k.shape[1], w, starts.data_ptr(),
            k_starts.data_ptr(), starts.shape[0] - 1, 1 if causal else 0,
            w ** -0.5 if scale is None else scale)


def _attend_checks(q, k, v, starts, k_starts):
    torch = _T().torch
    dev = _device_of(q, "q")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise EmeansError(f"EDTYPE: q {q.dtype} not supported (bfloat16 or float16)")
    _, hq, w, _, _ = _heads(q, dev, "q")
    nk, hk, wk, _, _ = _heads(k, dev, "k", q.dtype)
    nv, hv, wv, _, _ = _heads(v, dev, "v", q.dtype)
    if wk != w or (nv, hv, wv) != (nk, hk, wk):
        raise EmeansError(f"EINVAL: k and v must be rows x heads x {w} of one shape (got "
                          f"{tuple(k.shape)} and {tuple(v.shape)})")
    if w < 8 or w > 128 or w % 8:
        raise EmeansError(f"EINVAL: width must be a multiple of 8 in [8, 128] (got {w})")
    if hq < 1 or hk < 1 or hq % hk:
        raise EmeansError(f"EINVAL: {hq} heads of q cannot share {hk} of k and v")
    seqs = _vector(starts, dev, "starts", None, (torch.int32,), "int32") - 1
    if seqs < 0:
        raise EmeansError("EINVAL: starts must be one more than the sequences")
    if k_starts is not starts:
        _vector(k_starts, dev, "k_starts", seqs + 1, (torch.int32,), "int32")
    return dev


def _attend(q, k, v, starts, k_starts, causal, scale, keep):
    dev = _attend_checks(q, k, v, starts, k_starts)
    args = _attend_list(q, k, v, starts, k_starts, causal, scale)

    def call(st):
        torch, shape = _T().torch, q.shape
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
        lse = rest = None
        if keep:  # what the gradients need
            lse = torch.empty((shape[1], shape[0]), dtype=torch.float32, device=q.device)
            rest = torch.empty_like(out)
        _check(lib().emeans_attend(*args, out.data_ptr(), _ptr(lse), _ptr(rest), st))
        return out, lse, rest

    return _run(dev, None, call)


_attend_function = None


def _attend_fn():
    global _attend_function
    if _attend_function is None:
        torch = _T().torch

        class Attend(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, starts, k_starts, causal, scale):
                out, lse, rest = _attend(q, k, v, starts, k_starts, causal, scale, True)
                ctx.save_for_backward(q, k, v, starts, k_starts, out, lse, rest)
                ctx.args = causal, scale
                return out

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dout):
                q, k, v, starts, k_starts, out, lse, rest = ctx.saved_tensors
                args = _attend_list(q, k, v, starts, k_starts, *ctx.args)
                L, dtype, device, shape = lib(), q.dtype, q.device, q.shape

                def call(st):
                    g = _aligned(dout)
                    dq, dk, dv = (torch.empty(x.shape, dtype=dtype, device=device) for x in (q, k, v))
                    work = _work(L.emeans_attend_work(shape[0], k.shape[0], shape[1], k.shape[1],
                                                      shape[2], starts.shape[0] - 1), device)
                    _check(L.emeans_attend_gradient(
                        *args, out.data_ptr(), lse.data_ptr(), rest.data_ptr(), g.data_ptr(),
                        g.stride(0), g.stride(1), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                        _ptr(work), st))
                    return dq, dk, dv

                return *_run(q.get_device(), None, call), None, None, None, None

        _attend_function = Attend
    return _attend_function


def attend(q, k, v, starts, *, k_starts=None, causal: bool = True, scale=None, stream=None):
    """Attention over packed sequences of different lengths: q (n x hq x width), k and v
    (nk x hk x width; bfloat16 or float16), hk dividing hq; query head h reads key-value
    head h // (hq // hk). Sequence s is rows starts[s] .. starts[s + 1] (int32, one more
    than sequences, not decreasing) of q, and of k and v too or, where the keys are more
    or fewer than the queries, k_starts[s] .. k_starts[s + 1] of these. Returns
    softmax(scale q k^T) v, n x hq x width of q's type; scale is 1 / sqrt(width) by
    default, width a multiple of 8 up to 128.

    causal: of lq queries and lk keys of a sequence, query i sees keys j <= i + lk - lq
    (the last sees them all); otherwise every query sees all. Rows that see no key, and
    rows outside every sequence, are zeros. What a row does not see does not show in it,
    a NaN neither. The host reads no lengths, so the call may be captured.

    q, k and v have gradients (once: tangents of the forward mode are refused), sums in
    one order; a NaN may show anywhere in its sequence's gradients. Rows or heads that
    do not start at multiples of 16 bytes are copied first."""
    _device_of(q, "q")
    if stream is not None:
        with _T().torch.cuda.stream(stream):
            return attend(q, k, v, starts, k_starts=k_starts, causal=causal, scale=scale)
    _no_tangent("attend", q, k, v)
    if any(t.dim() != 3 for t in (q, k, v)):
        raise EmeansError("EINVAL: q, k and v must be rows x heads x width")
    if k_starts is None:
        if k.shape[0] != q.shape[0]:
            raise EmeansError(f"EINVAL: k and v must have the {q.shape[0]} rows of q, or k_starts be "
                              "given")
        k_starts = starts
    q, k, v = _aligned(q), _aligned(k), _aligned(v)
    if _T().torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        return _attend_fn().apply(q, k, v, starts, k_starts, causal, scale)
    return _attend(q, k, v, starts, k_starts, causal, scale, False)[0]


def _paged(dev, store, block, what):
    """(codes, scales) of a paged store: its format, row length and shape."""
    if not isinstance(store, (tuple, list)) or len(store) != 2:
        raise EmeansError(f"EINVAL: {what} must be (codes, scales)")
    fmt, _, d = _store(dev, store[0], store[1], block)
    if store[0].dim() != 3:
        raise EmeansError(f"EINVAL: codes of {what} must be pages x page rows x d")
    return fmt, d, store[0].shape


def _places(dev, table, lengths, page: int):
    """Sequences, table entries of one, the table's row distance and the places
    that a sequence has at most."""
    t = _T().torch
    seqs, pages, ld = _matrix(table, dev, "table", (t.int32,), "int32")
    _vector(lengths, dev, "lengths", seqs, (t.int32,), "int32")
    return seqs, pages, ld, pages * page


def cache_attend(q, keys, values, table, lengths, *, block: int = BLOCK, scale=None, weights=None,
                 stream=None):
    """Attention of one new token per sequence over a paged store: q (seqs x hq x
    width; float32, bfloat16 or float16), keys and values each (codes, scales) of
    cache_new((pages, page rows), hk * width, block=block), hk dividing hq; query head
    h reads key-value head h // (hq // hk). Sequence s is the first lengths[s] (int32)
    places of its row of `table` (seqs x pages int32, as cache_read_pages takes it;
    places in pages outside the store are left out, lengths cut to what the table
    holds). Returns seqs x hq x width of q's type, zeros for a sequence without places.
    scale: of q.k, 1 / sqrt(width) by default. width is a multiple of 16 up to 128.

    weights: a float32 tensor seqs x places (places = the table's columns x page
    rows) to whose row s the softmax weights of each place, summed over the heads, are
    added: what cache_evict goes by.

    The time goes by the table's columns too: pass table[:, :m] where m pages hold
    every sequence. There is no gradient (`attend` is for training): where gradients are
    enabled, a q or weights that ask for one are refused."""
    dev = _device_of(q, "q")
    dt = _number(q.dtype, "q")
    _no_gradient("cache_attend", q)
    seqs, hq, width, qr, qh = _heads(q, dev, "q")
    fmt, d, shape = _paged(dev, keys, block, "keys")
    vfmt, _, vshape = _paged(dev, values, block, "values")
    if vfmt != fmt or vshape != shape:
        raise EmeansError("EINVAL: keys and values must be stores of one shape and format")
    if width < 16 or width > 128 or width % 16 or d % width or not d:
        raise EmeansError(f"EINVAL: width must be a multiple of 16 in [16, 128] that divides the "
                          f"store's rows of {d} (got {width})")
    hk = d // width
    if hq < 1 or hq % hk:
        raise EmeansError(f"EINVAL: {hq} heads of q cannot share {hk} of the store")
    n, pages, ld, places = _places(dev, table, lengths, shape[1])
    if n != seqs:
        raise EmeansError(f"EINVAL: table must have a row for each of the {seqs} rows of q")
    wld = 0
    if weights is not None:
        torch = _T().torch
        wn, wd, wld = _matrix(weights, dev, "weights", (torch.float32,), "float32")
        _no_gradient("cache_attend", weights)
        if (wn, wd) != (seqs, places) or (wld < places and seqs > 1):
            raise EmeansError(f"EINVAL: weights must be {seqs} x {places}")

    def call(st):
        out = _T().torch.empty((seqs, hq, width), dtype=q.dtype, device=q.device)
        if seqs:
            L = lib()
            with_weights = 1 if weights is not None else 0
            work = _work(L.emeans_cache_attend_work(seqs, hq, hk, width, shape[1], pages,
                                                    with_weights), q.device)
            _check(L.emeans_cache_attend(
                q.data_ptr(), dt, qr, qh, keys[0].data_ptr(), keys[1].data_ptr(),
                values[0].data_ptr(), values[1].data_ptr(), shape[0], shape[1], block, fmt,
                table.data_ptr(), ld, pages, lengths.data_ptr(), seqs, hq, hk, width,
                width ** -0.5 if scale is None else scale, out.data_ptr(),
                weights.data_ptr() if with_weights and places else None, wld, _ptr(work), st))
        return out

    return _run(dev, stream, call)


def cache_evict(stores, table, lengths, weights, keep: int, *, recent: int = 0, block: int = BLOCK,
                stream=None):
    """Drop rows of small weight from one to four paged stores of one page layout
    ((codes, scales) each, none of them twice: keys and values, say): of a sequence of more than `keep`
    rows stay the last `recent` and, of those before them, the keep - recent of
    largest weight (weights: seqs x places float32, as cache_attend adds them up; of
    equal ones the first, NaN counts as -infinity). They move to the sequence's first
    places in their order, in place; the pages behind them are free.

    table and lengths as for cache_attend, lengths and weights unchanged; no page may
    be in use twice (its rows would be moved for each use). Returns (lengths, weights,
    kept): the new lengths (int32), the weights of the rows that stayed at their new
    places and zeros behind them, and the places they came from (seqs x keep int32, -1
    behind the last)."""
    if not isinstance(stores, (tuple, list)) or not 1 <= len(stores) <= 4:
        raise EmeansError("EINVAL: stores must be one to four (codes, scales)")
    keep, recent = int(keep), int(recent)
    dev = _device_of(lengths, "lengths")
    found = [_paged(dev, s, block, "stores") for s in stores]
    shape = found[0][2]
    if any(f[2][:2] != shape[:2] for f in found) or not all(f[1] for f in found):
        raise EmeansError("EINVAL: the stores must have the same pages of rows")
    if shape[0] and len({s[0].data_ptr() for s in stores}) < len(stores):
        raise EmeansError("EINVAL: a store is given twice")
    seqs, pages, ld, places = _places(dev, table, lengths, shape[1])
    torch = _T().torch
    wn, wd, wld = _matrix(weights, dev, "weights", (torch.float32,), "float32")
    if (wn, wd) != (seqs, places) or (wld < places and seqs > 1):
        raise EmeansError(f"EINVAL: weights must be {seqs} x {places}")
    _no_gradient("cache_evict", weights)
    if not 0 <= keep < 2 ** 31 - 1023 or not 0 <= recent <= keep:
        raise EmeansError(f"EINVAL: keep or recent out of range ({keep}, {recent})")

    def call(st):
        empty, device = torch.empty, codes[0].device
        new = empty((seqs,), dtype=torch.int32, device=device)
        new_weights = empty((seqs, places), dtype=torch.float32, device=device)
        kept = empty((seqs, keep), dtype=torch.int32, device=device)
        if seqs:
            L, m = lib(), len(stores)
            work = _work(L.emeans_cache_evict_work(seqs, keep if keep < places else 0), device)
            _check(L.emeans_cache_evict(
                (c_vp * m)(*(t.data_ptr() for t in codes)),
                (c_vp * m)(*(t.data_ptr() for t in scales)),
                (c_i64 * m)(*(t.shape[2] for t in codes)),
                (c_i64 * m)(*(t.shape[2] for t in scales)), m, shape[0], shape[1],
                table.data_ptr(), ld, pages, lengths.data_ptr(), seqs, weights.data_ptr(), wld,
                keep, recent, new.data_ptr(), new_weights.data_ptr(), kept.data_ptr(), _ptr(work),
                st))
        return new, new_weights, kept

    codes, scales = [s[0] for s in stores], [s[1] for s in stores]
    return _run(dev, stream, call)


def batch_rows(n: int, seed: int, pass_: int, start: int, count: int, device="cuda", stream=None):
    """Rows visited by slots [start, start+count) of a pass of a training run
    (pass_ = -1: the order whose first k entries are train()'s starting rows)."""
    import torch
    out = torch.empty((count,), dtype=torch.int32, device=device)
    with torch.cuda.device(out.device):
        s = stream if stream is not None else torch.cuda.current_stream(out.device)
        if count:
            _check(lib().emeans_batch_rows(int(n), int(seed) & (2**64 - 1), int(pass_),
                                           int(start), int(count), out.data_ptr(),
                                           ctypes.c_void_p(s.cuda_stream)))
    return out


class Stream:
    """Streaming training (README "Data too big for memory"): the step loop of
    train() with the rows supplied by the caller, for data that stays off the
    device. The model (centroids and running statistics) lives on the device
    of the start centroids. Pass e takes recipe["epoch_rows"][e] rows in
    batches of recipe["batch_size"] rows (the pass's last batch holds the
    rest); each batch goes in through one or more accumulate() calls followed
    by one update(), and end_epoch() closes the pass. finalize() returns the
    centroids; final_closing_mean() may first replace the closing statistics
    with a second look at the rows. All library work runs on `stream` (the
    current stream of the start centroids' device by default)."""

    def __init__(self, n: int, start, T: float = 5.0, seed: int = 1234, *, dtype=None,
                 batch_law="auto", batch_size: int = 0, alpha0: float = 0.0,
                 unused_threshold=None, finalize: bool = True, bf16_search: bool = False,
                 spherical: bool = False, profile: bool = False, counts: bool = False,
                 split_log_cap: int = 0, slow_ema: float = 0.0, search=None, search_shift=None,
                 search_scale=None, stream=None):
        import torch
        if not (getattr(start, "is_cuda", False) and start.dtype == torch.float32
                and start.is_contiguous() and start.dim() == 2):
            raise EmeansError("EINVAL: start must be a contiguous k x d float32 tensor on the GPU")
        self.k, self.d = start.shape
        self.n = int(n)
        self.device = start.device
        codes = {None: F32, torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8,
                 torch.float8_e4m3fn: F8, torch.float16: F16, torch.uint8: U8}
        code = codes.get(dtype, -1)
        if code < 0:
            raise EmeansError(f"EDTYPE: {dtype} not supported (float32, bfloat16, float16, int8, "
                              f"uint8 or float8_e4m3fn)")
        self.dtype = {F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8,
                      F8: torch.float8_e4m3fn, F16: torch.float16, U8: torch.uint8}[code]
        self._stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        with torch.cuda.device(self.device):
            o = _opts(code, batch_law, batch_size, alpha0, unused_threshold, finalize, profile,
                      ctypes.c_void_p(self._stream.cuda_stream))
            o.bf16_search = 1 if bf16_search else 0
            o.spherical = 1 if spherical else 0
            _set_search(o, search, search_shift, search_scale, self.d)
            self._search_shift = search_shift   # read by the library until close()
            self._counts = torch.empty((self.k,), dtype=torch.float32, device=self.device) \
                if counts else None
            self._log = (ctypes.c_int32 * (3 * split_log_cap))() if split_log_cap > 0 else None
            if self._counts is not None:
                o.out_counts = self._counts.data_ptr()
            if self._log is not None:
                o.split_log = ctypes.cast(self._log, c_vp)
                o.split_log_cap = split_log_cap
            # the slow-EMA centroids (slow_ema) are written by finalize()
            self.slow_centroids = torch.empty((self.k, self.d), dtype=torch.float32,
                                              device=self.device) if slow_ema else None
            if self.slow_centroids is not None:
                o.slow_ema = float(slow_ema)
                o.slow_centroids = self.slow_centroids.data_ptr()
            self._opts = o
            self.recipe = recipe(self.n, self.d, self.k, T, batch_law=batch_law,
                                 batch_size=batch_size, alpha0=alpha0,
                                 unused_threshold=unused_threshold)
            h = c_vp()
            _check(lib().emeans_begin(self.n, self.d, self.k, float(T), int(seed) & (2**64 - 1),
                                      start.data_ptr(), ctypes.byref(o), ctypes.byref(h)))
            self._h = h
        self.stats = None

    def _handle(self):
        if self._h is None or not self._h.value:
            raise EmeansError("EINVAL: the model was closed")
        return self._h

    def accumulate(self, batch, labels: bool = True):
        """Add a batch (or a piece of one); returns its labels (int32) or None."""
        import torch
        _require_device(batch)
        if batch.dtype != self.dtype or batch.dim() != 2 or batch.shape[1] != self.d:
            raise EmeansError(f"EINVAL: batch must be rows x {self.d} {self.dtype}")
        with torch.cuda.stream(self._stream):   # allocated where the library writes it
            out = torch.empty((batch.shape[0],), dtype=torch.int32, device=self.device) \
                if labels else None
        _check(lib().emeans_accumulate(self._handle(), batch.data_ptr(), int(batch.shape[0]),
                                       out.data_ptr() if out is not None else None))
        return out

    def update(self, _accumulated=None) -> None:
        _check(lib().emeans_update(self._handle()))

    def end_epoch(self) -> None:
        _check(lib().emeans_end_epoch(self._handle()))

    def final_closing_mean(self, batches, assignments=None, labels_out: bool = False):
        """Replace the closing statistics with a second look at the rows
        (README "Several GPUs", final_closing_mean), after the last
        end_epoch() and before finalize().

        batches: device tensors (rows x d, the model's dtype, row-major) that
        together go over the rows in one fixed order. assignments: None, or
        one label per row in that same order (int32 or int64, host or device;
        -1 for a row the last pass skipped): the labels kept from the final
        pass, so that no search is needed. Without them every row is assigned
        once more against the final EMA centroids. Blocks larger than the
        batch size are sent in pieces. finalize() then gives each centroid the
        exact mean of the rows counted under it (the EMA centroid where none
        was). With labels_out, returns the labels used (int32, device, the
        concatenation over the batches)."""
        import torch
        B = int(self.recipe["batch_size"])
        lab_all = None
        if assignments is not None:
            lab_all = torch.as_tensor(assignments)
            if lab_all.dim() != 1 or lab_all.dtype not in (torch.int32, torch.int64):
                raise EmeansError("EINVAL: assignments must be one int32 or int64 label per row")
        used = []
        pos = 0
        with torch.cuda.device(self.device), torch.cuda.stream(self._stream):
            for batch in batches:
                _require_device(batch)
                if (batch.dtype != self.dtype or batch.dim() != 2 or batch.shape[1] != self.d
                        or not batch.is_contiguous()):
                    raise EmeansError(f"EINVAL: batches must be contiguous rows x {self.d} "
                                      f"{self.dtype} tensors")
                m = int(batch.shape[0])
                for a in range(0, m, B):
                    piece = batch[a:a + B]
                    nb = int(piece.shape[0])
                    lab = None
                    if lab_all is not None:
                        if pos + a + nb > lab_all.numel():
                            raise EmeansError("EINVAL: assignments hold fewer labels than the "
                                              "batches have rows")
                        lab = lab_all[pos + a:pos + a + nb].to(self.device, torch.int32)
                    out = torch.empty((nb,), dtype=torch.int32, device=self.device) \
                        if labels_out else None
                    _check(lib().emeans_closing_add(
                        self._handle(), piece.data_ptr(), nb,
                        lab.data_ptr() if lab is not None else None,
                        out.data_ptr() if out is not None else None))
                    if out is not None:
                        used.append(out)
                pos += m
        if lab_all is not None and pos != lab_all.numel():
            raise EmeansError("EINVAL: assignments hold more labels than the batches have rows")
        if labels_out:
            return torch.cat(used) if used else torch.zeros(0, dtype=torch.int32,
                                                             device=self.device)
        return None

    def finalize(self):
        """Centroids (k x d float32): the closing mean once every pass ended."""
        import torch
        C = torch.empty((self.k, self.d), dtype=torch.float32, device=self.device)
        s = Stats()
        _check(lib().emeans_finalize(self._handle(), C.data_ptr(), ctypes.byref(s)))
        self.stats = _stats_dict(s)
        return C

    @property
    def counts(self):
        return self._counts

    @property
    def split_log(self):
        if self._log is None or self.stats is None:
            return None
        m = self.stats["n_splits"] if self.stats["n_splits"] < len(self._log) // 3 else len(self._log) // 3
        return [tuple(self._log[3 * i:3 * i + 3]) for i in range(m)]

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().emeans_free(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def begin(n: int, start, T: float = 5.0, seed: int = 1234, **kw) -> Stream:
    return Stream(n, start, T, seed, **kw)


@dataclass
class HostTrainOutput:
    centroids: object          # k x d float32 tensor
    labels: object             # n int32 numpy array (last pass) or None
    stream: "Stream"
    trace: object = None       # every batch's labels in step order (int32 numpy) or None


def train_from_host(Xh, k: int, T: float = 5.0, seed: int = 1234, *, start=None,
                    labels: bool = True, trace: bool = False, order=None, device="cuda",
                    **kw) -> HostTrainOutput:
    """Train on a host array (numpy, row-major n x d float32, e.g. a memory
    map) that need not fit on the device, through a Stream model.

    Visiting order: order(e, rows) gives the host row ids of pass e; by
    default the library's own sampler (batch_rows), i.e. the very rows
    emeans_train visits with this seed. Starting centroids: `start` (k x d
    float32 on the device), by default the rows emeans_train starts from
    (batch_rows with pass -1). With both defaults a host run sees the same
    batches as train() on resident data.

    Transfer: each batch is gathered on the host into one of two pinned
    buffers, which take turns; a copy stream moves it to the device while
    the model's stream still computes on the other one. One event per buffer
    says the copy has landed, another that the model is done reading it
    (both streams keep the default priority)."""
    import numpy as np
    import torch
    Xh = np.asarray(Xh)
    if Xh.dtype != np.float32 or Xh.ndim != 2:
        raise EmeansError("EINVAL: Xh must be an n x d float32 array")
    n, d = Xh.shape
    dev = torch.device(device)
    if start is None:
        first = batch_rows(n, seed, -1, 0, k, device=dev).cpu().numpy()
        start = torch.from_numpy(np.ascontiguousarray(Xh[first])).to(dev)
    if order is None:
        def order(e, rows):
            return batch_rows(n, seed, e, 0, rows, device=dev).cpu().numpy()
    em = Stream(n, start, T, seed, **kw)
    B = int(em.recipe["batch_size"])
    passes = em.recipe["epoch_rows"]
    # (pass, host rows) of every update step, in schedule order
    steps = [(e, ids[a:a + B]) for e, rows_e in enumerate(passes)
             for ids in [np.asarray(order(e, rows_e))] for a in range(0, rows_e, B)]
    host = [torch.empty((B, d), dtype=torch.float32).pin_memory() for _ in range(2)]
    staged = [torch.empty((B, d), dtype=torch.float32, device=dev) for _ in range(2)]
    mover = torch.cuda.Stream(device=dev)
    landed = [torch.cuda.Event() for _ in range(2)]
    released = [torch.cuda.Event() for _ in range(2)]
    for ev in released:
        ev.record(em._stream)

    def send(j):
        """Gather step j's rows into buffer j % 2 and queue its upload."""
        buf = j % 2
        ids = steps[j][1]
        released[buf].synchronize()      # the model no longer reads this buffer
        np.take(Xh, ids, axis=0, out=host[buf].numpy()[:len(ids)])
        mover.wait_event(released[buf])
        with torch.cuda.stream(mover):
            staged[buf][:len(ids)].copy_(host[buf][:len(ids)], non_blocking=True)
        landed[buf].record(mover)

    final = len(passes) - 1
    kept = []                              # (pass, rows, device labels)
    if steps:
        send(0)
    for j, (e, ids) in enumerate(steps):
        buf = j % 2
        if j + 1 < len(steps):
            send(j + 1)                  # the next upload overlaps this step
        em._stream.wait_event(landed[buf])
        want = trace or (labels and e == final)
        lab = em.accumulate(staged[buf][:len(ids)], labels=want)
        released[buf].record(em._stream)
        em.update()
        if lab is not None:
            kept.append((e, ids, lab))
        if j + 1 == len(steps) or steps[j + 1][0] != e:
            em.end_epoch()
    C = em.finalize()                    # synchronises the model's stream
    out_labels = np.full(n, -1, dtype=np.int32) if labels else None
    tr = []
    for e, ids, lab in kept:
        h = lab.cpu().numpy()
        if labels and e == final:
            out_labels[ids] = h
        if trace:
            tr.append(h)
    return HostTrainOutput(C, out_labels, em, np.concatenate(tr) if trace and tr else None)
