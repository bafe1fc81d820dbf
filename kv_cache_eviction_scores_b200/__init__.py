"""DropKV prefill-time KV-cache eviction scoring on NVIDIA B200 (sm_100a).

A thin ctypes binding over ``libdropkv.so`` (C ABI: ``include/dropkv.h``).
It only marshals arguments: PyTorch supplies device memory and the current
stream, and every step of the scoring path runs in the library's CUDA kernels.
There is no CPU fallback; without the built library every call raises.

What is scored (write-up "DropKV：精确单项输出扰动评分组件", section 核心公式
and the Algorithm 1 paragraph): for the last ``window`` prompt queries,
p = softmax(K q / sqrt d), a = sum_j p_j v_j, Delta_j = p_j/(1-p_j) (a - v_j),
s_j = sum_t ||Delta_j||^2; scores are averaged over the query heads of each KV
head, max-pooled, the window is set to +inf, and the lowest scores are evicted.

Usage (CUDA tensors; q holds the last ``window`` query rows of each sequence)::

    import kv_cache_eviction_scores_b200 as dk
    # q [B, Hq, window, d], k / v [B, Hkv, n_max, d], bf16 or fp32
    scores = dk.dropkv_scores(q, k, v, window, pool_kernel, lengths)   # [B, Hkv, n_max]
    keep_idx, evict_idx = dk.dropkv_select(scores, keep_counts, lengths)
    # or both at once:
    scores, keep_idx, evict_idx = dk.evict(q, k, v, window, pool_kernel, keep_counts, lengths)
    # the attention-only control score through the same pipeline:
    control = dk.dropkv_scores(q, k, v, window, pool_kernel, lengths, score="attention")

The kept rows, and the tokens after them, live in a paged cache (bf16, fp32, or
e4m3 with a power-of-two scale per row)::

    # pages [n_pages, Hkv, page_size, d], page_table int32 [B, max_pages]
    dk.dropkv_cache_write(k, v, k_pages, v_pages, page_table, rows=keep_idx)   # kept -> slots 0..
    dk.dropkv_cache_write(k_new, v_new, k_pages, v_pages, page_table, start=lengths)  # append
    # q [B, Hq, T, d]: the last T of each sequence's `lengths` slots
    out = dk.dropkv_cache_attention(q, k_pages, v_pages, page_table, lengths)
    k, v = dk.dropkv_cache_read(k_pages, v_pages, page_table, n)               # back to dense
    # an eviction whose kept rows go straight into a cache:
    dk.evict_to_cache(q, k, v, window, pool_kernel, keep_counts, k_pages, v_pages, page_table)
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Sequence, Tuple

import torch

__all__ = [
    "DropKVError", "SingularError", "Shape", "Options", "lib", "lib_path",
    "make_shape", "scores_workspace_bytes", "select_workspace_bytes", "dropkv_scores",
    "dropkv_select", "evict", "evict_to_cache", "dropkv_cache_write", "dropkv_cache_read",
    "dropkv_cache_attention", "cache_attention_workspace", "cache_attention_workspace_bytes",
    "cache_attention_path",
    "Cache", "CacheRows", "CacheAttn", "auto_path", "scores_launches", "select_launches",
    "selftest_wait_timeout", "selftest_select_timeout", "selftest_cache_attention_timeout",
    "OK", "ERR_ARG", "ERR_SINGULAR", "ERR_CUDA", "ERR_UNSUPPORTED", "ERR_WORKSPACE", "ERR_TIMEOUT",
    "PATH_AUTO", "PATH_SIMT", "PATH_TENSOR", "SCORE_PERTURBATION", "SCORE_ATTENTION",
]

OK, ERR_ARG, ERR_SINGULAR, ERR_CUDA, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_TIMEOUT = range(7)
PATH_AUTO, PATH_SIMT, PATH_TENSOR = 0, 1, 2
_PATHS = {"auto": PATH_AUTO, "simt": PATH_SIMT, "tensor": PATH_TENSOR}
SCORE_PERTURBATION, SCORE_ATTENTION = 0, 1
_SCORES = {"perturbation": SCORE_PERTURBATION, "attention": SCORE_ATTENTION}
BF16, F32, E4M3 = 0, 1, 2
_PAGE_DTYPES = {torch.bfloat16: BF16, torch.float32: F32, torch.float8_e4m3fn: E4M3}
_DENSE_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libdropkv.so")


class DropKVError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = _status_string(status)
        super().__init__(f"{what}: {msg} (status {status})" if what else msg)


class SingularError(DropKVError):
    """Some window probability rounds to 1: exact single removal is undefined."""


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "Hq", "Hkv", "n_max", "d", "window", "pool_kernel", "dtype")]


class Options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("score", ctypes.c_int32),
                ("attn_out", ctypes.c_void_p), ("stats_out", ctypes.c_void_p),
                ("events", ctypes.c_void_p), ("n_events", ctypes.c_int32),
                ("tc_ctas", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "Hkv", "d", "n_pages", "page_size", "max_pages", "dtype", "reserved")] + \
               [(n, ctypes.c_void_p) for n in
                ("k_pages", "v_pages", "k_scale", "v_scale", "page_table")]


class CacheRows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("dtype", ctypes.c_int32), ("n", ctypes.c_int32), ("m", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("rows", ctypes.c_void_p),
                ("start", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


class CacheAttn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3),
                ("dtype", ctypes.c_int32), ("Hq", ctypes.c_int32), ("T", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("path", ctypes.c_int32),
                ("lengths", ctypes.c_void_p), ("q_lengths", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libdropkv.so (built in-tree by ``python -m kv_cache_eviction_scores_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libdropkv.so is not built ({path}); run "
                           "`python -m kv_cache_eviction_scores_b200.build`")
    L = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    ip = ctypes.POINTER(ctypes.c_int32)
    sp = ctypes.POINTER(Shape)
    L.dropkv_scores_workspace_bytes.argtypes = [sp]
    L.dropkv_scores_workspace_bytes.restype = sz
    L.dropkv_scores.argtypes = [sp, vp, vp, vp, ip, vp, vp, sz, vp]
    L.dropkv_scores.restype = i32
    L.dropkv_scores_async.argtypes = [sp, vp, vp, vp, ip, vp, vp, sz, vp, vp]
    L.dropkv_scores_async.restype = i32
    L.dropkv_scores_ex.argtypes = [sp, vp, vp, vp, ip, vp, vp, sz, vp, vp,
                                   ctypes.POINTER(Options)]
    L.dropkv_scores_ex.restype = i32
    L.dropkv_select_workspace_bytes.argtypes = [i32, i32, i32]
    L.dropkv_select_workspace_bytes.restype = sz
    L.dropkv_select.argtypes = [i32, i32, i32, vp, ip, ip, vp, i32, vp, i32, vp, sz, vp]
    L.dropkv_select.restype = i32
    L.dropkv_select_ex.argtypes = [i32, i32, i32, vp, ip, ip, vp, i32, vp, i32, vp, sz, vp, vp]
    L.dropkv_select_ex.restype = i32
    L.dropkv_auto_path.argtypes = [sp]
    L.dropkv_auto_path.restype = i32
    L.dropkv_scores_launches.argtypes = [sp, ip, i32]
    L.dropkv_scores_launches.restype = i32
    L.dropkv_select_launches.argtypes = [i32, i32, i32, ip]
    L.dropkv_select_launches.restype = i32
    L.dropkv_scores_select.argtypes = [sp, vp, vp, vp, ip, ip, vp, vp, i32, vp, i32, vp, sz, vp,
                                       vp, ctypes.POINTER(Options)]
    L.dropkv_scores_select.restype = i32
    L.dropkv_scores_select_launches.argtypes = [sp, ip, i32]
    L.dropkv_scores_select_launches.restype = i32
    L.dropkv_status_string.argtypes = [i32]
    L.dropkv_status_string.restype = ctypes.c_char_p
    L.dropkv_abi_version.argtypes = []
    L.dropkv_abi_version.restype = i32
    L.dropkv_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint64, vp]
    L.dropkv_selftest_wait_timeout.restype = i32
    L.dropkv_selftest_select_timeout.argtypes = [i32, i32, i32, vp, ip, ip, vp, i32, vp, i32, vp,
                                                 ctypes.c_uint64, vp]
    L.dropkv_selftest_select_timeout.restype = i32
    L.dropkv_last_cuda_error.argtypes = []
    L.dropkv_last_cuda_error.restype = i32
    L.dropkv_last_cuda_error_string.argtypes = []
    L.dropkv_last_cuda_error_string.restype = ctypes.c_char_p
    cp, rp, ap = ctypes.POINTER(Cache), ctypes.POINTER(CacheRows), ctypes.POINTER(CacheAttn)
    for fn in (L.dropkv_cache_write, L.dropkv_cache_read):
        fn.argtypes = [cp, rp, vp, vp]
        fn.restype = i32
    L.dropkv_cache_attention_workspace_bytes.argtypes = [cp, ap]
    L.dropkv_cache_attention_workspace_bytes.restype = sz
    L.dropkv_cache_attention.argtypes = [cp, ap, vp, sz, vp, vp]
    L.dropkv_cache_attention.restype = i32
    L.dropkv_cache_attention_path.argtypes = [cp, ap]
    L.dropkv_cache_attention_path.restype = i32
    L.dropkv_selftest_cache_attention_timeout.argtypes = [cp, ap, vp, sz, vp, ctypes.c_uint64, vp]
    L.dropkv_selftest_cache_attention_timeout.restype = i32
    _lib = L
    return L


def _status_string(status: int) -> str:
    try:
        return lib().dropkv_status_string(status).decode()
    except Exception:
        return f"status {status}"


def _check(status: int, what: str):
    if status == OK:
        return
    if status == ERR_SINGULAR:
        raise SingularError(status, what)
    if status == ERR_CUDA:
        what = f"{what} [{lib().dropkv_last_cuda_error_string().decode()}]"
    raise DropKVError(status, what)


def _i32_array(vals: Optional[Sequence[int]]):
    if vals is None:
        return None
    arr = (ctypes.c_int32 * len(vals))(*[int(x) for x in vals])
    return arr


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


# The current stream's handle without a torch.cuda.Stream around it (2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def make_shape(q: torch.Tensor, k: torch.Tensor, window: int, pool_kernel: int) -> Shape:
    B, Hq, w, d = q.shape
    Bk, Hkv, n_max, dk = k.shape
    if (B, d) != (Bk, dk) or w != window:
        raise ValueError("q must be [B, Hq, window, d] and k, v [B, Hkv, n_max, d]")
    if q.dtype == torch.bfloat16:
        dt = BF16
    elif q.dtype == torch.float32:
        dt = F32
    else:
        raise TypeError("q, k, v must be bfloat16 or float32")
    return Shape(B, Hq, Hkv, n_max, d, window, pool_kernel, dt)


def scores_workspace_bytes(shape: Shape) -> int:
    return int(lib().dropkv_scores_workspace_bytes(ctypes.byref(shape)))


def select_workspace_bytes(B: int, Hkv: int, n_max: int) -> int:
    return int(lib().dropkv_select_workspace_bytes(B, Hkv, n_max))


def auto_path(shape: Shape) -> int:
    return int(lib().dropkv_auto_path(ctypes.byref(shape)))


def scores_launches(shape: Shape, lengths=None, path: str = "auto") -> int:
    return int(lib().dropkv_scores_launches(ctypes.byref(shape), _i32_array(lengths),
                                            _PATHS[path]))


def select_launches(B: int, Hkv: int, n_max: int, lengths=None) -> int:
    return int(lib().dropkv_select_launches(B, Hkv, n_max, _i32_array(lengths)))


def scores_select_launches(shape: Shape, lengths=None, path: str = "auto") -> int:
    return int(lib().dropkv_scores_select_launches(ctypes.byref(shape), _i32_array(lengths),
                                                   _PATHS[path]))


def _check_inputs(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor (there is no CPU path)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share one dtype")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k and v must be on one device")


def dropkv_scores(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int,
                  pool_kernel: int, lengths: Optional[Sequence[int]] = None, *,
                  path: str = "auto", out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, return_attn: bool = False,
                  status: Optional[torch.Tensor] = None, kernel_events=None,
                  score: str = "perturbation", tc_ctas: int = 0):
    """fp32 scores [B, Hkv, n_max] (pooled, window = +inf, padding = NaN).

    q: [B, Hq, window, d] window queries; k, v: [B, Hkv, n_max, d]; lengths:
    per-row lengths (host ints) or None for n_max.  With ``status`` (a CUDA
    int32 tensor of one element) the call is asynchronous and the singular flag
    lands there; otherwise it synchronises and raises SingularError.
    With ``return_attn`` also returns the window attention outputs
    [B, Hq, window, d] and (max logit, normaliser) stats [B, Hq, window, 2].
    ``kernel_events``: torch.cuda.Event objects (each recorded once already so
    that its handle exists); events 2i / 2i+1 bracket the i-th kernel launch.
    ``score``: "perturbation" (DropKV's exact single-removal score) or
    "attention" (the accumulated window attention probability, the control
    score), same merge / pool / window handling.
    ``tc_ctas``: on the tensor path, the most CTAs a scoring pass launches
    (0 = one per SM); fewer CTAs walk longer runs of tiles each.
    """
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    _check_inputs(q, k, v)
    shape = make_shape(q, k, window, pool_kernel)
    dev = q.device
    if out is None:
        out = torch.empty(shape.B, shape.Hkv, shape.n_max, dtype=torch.float32, device=dev)
    need = scores_workspace_bytes(shape)
    if need == 0:
        raise DropKVError(ERR_ARG, "dropkv_scores_workspace_bytes")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    opts = Options(_PATHS[path], _SCORES[score], None, None, None, 0, int(tc_ctas))
    ev_arr = None
    if kernel_events:
        # raw cudaEvent_t handles of (already recorded once) torch.cuda.Event objects
        ev_arr = (ctypes.c_void_p * len(kernel_events))(*[e.cuda_event for e in kernel_events])
        opts.events = ctypes.cast(ev_arr, ctypes.c_void_p)
        opts.n_events = len(kernel_events)
    attn = stats = None
    if return_attn:
        attn = torch.empty(shape.B, shape.Hq, window, shape.d, dtype=torch.float32, device=dev)
        stats = torch.empty(shape.B, shape.Hq, window, 2, dtype=torch.float32, device=dev)
        opts.attn_out = attn.data_ptr()
        opts.stats_out = stats.data_ptr()
    st = lib().dropkv_scores_ex(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                _i32_array(lengths), _ptr(out), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(dev),
                                _ptr(status), ctypes.byref(opts))
    _check(st, "dropkv_scores")
    if return_attn:
        return out, attn, stats
    return out


def selftest_wait_timeout(limit_ms: float = 20.0, device=None) -> int:
    """Runs the bounded-wait self-test (a wait on an mbarrier nothing arrives
    on) and returns the status word it leaves: ERR_TIMEOUT when the device-side
    wait gave up as designed."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(lib().dropkv_selftest_wait_timeout(_ptr(status), int(limit_ms * 1e6), _stream(dev)),
           "dropkv_selftest_wait_timeout")
    torch.cuda.synchronize(dev)
    return int(status.item())


def selftest_select_timeout(scores: torch.Tensor, keep_counts: Sequence[int],
                            lengths: Optional[Sequence[int]] = None, limit_ms: float = 20.0):
    """Runs the select kernel with one CTA of every segment withholding an
    arrival and waits limited to ``limit_ms``; returns (status word, keep_idx,
    evict_idx).  Segments with evictions report ERR_TIMEOUT and lists of -1."""
    B, Hkv, n_max = scores.shape
    lens = list(lengths) if lengths is not None else [n_max] * B
    keep = [int(x) for x in keep_counts]
    max_keep = max(keep)
    max_evict = max(L - kc for L, kc in zip(lens, keep))
    dev = scores.device
    keep_idx = torch.full((B, Hkv, max_keep), 7, dtype=torch.int32, device=dev)
    evict_idx = torch.full((B, Hkv, max_evict), 7, dtype=torch.int32, device=dev)
    status = torch.full((1,), -1, dtype=torch.int32, device=dev)
    _check(lib().dropkv_selftest_select_timeout(
        B, Hkv, n_max, _ptr(scores), _i32_array(lengths), _i32_array(keep), _ptr(keep_idx),
        max_keep, _ptr(evict_idx), max_evict, _ptr(status), int(limit_ms * 1e6), _stream(dev)),
        "dropkv_selftest_select_timeout")
    torch.cuda.synchronize(dev)
    return int(status.item()), keep_idx, evict_idx


def dropkv_select(scores: torch.Tensor, keep_counts: Sequence[int],
                  lengths: Optional[Sequence[int]] = None, *, max_keep: Optional[int] = None,
                  max_evict: Optional[int] = None,
                  workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None,
                  sync: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keep / evict positions per (b, h), ascending, padded with -1 (int32).

    Asynchronous by default.  With ``status`` (a CUDA int32 tensor of one
    element) the device-side status of the kernels (OK, or ERR_TIMEOUT if a
    bounded wait gave up) lands there; with ``sync=True`` the call waits for
    the stream and raises on a device-side error.
    """
    if not scores.is_cuda or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise TypeError("scores must be a contiguous CUDA float32 tensor")
    B, Hkv, n_max = scores.shape
    lens = list(lengths) if lengths is not None else [n_max] * B
    keep = [int(x) for x in keep_counts]
    if len(keep) != B or len(lens) != B:
        raise ValueError("keep_counts and lengths need one entry per batch row")
    if max_keep is None:
        max_keep = max(keep)
    if max_evict is None:
        max_evict = max(L - kc for L, kc in zip(lens, keep))
    dev = scores.device
    keep_idx = torch.empty(B, Hkv, max_keep, dtype=torch.int32, device=dev)
    evict_idx = torch.empty(B, Hkv, max_evict, dtype=torch.int32, device=dev)
    need = select_workspace_bytes(B, Hkv, n_max)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    args = (B, Hkv, n_max, _ptr(scores), _i32_array(lengths), _i32_array(keep), _ptr(keep_idx),
            max_keep, _ptr(evict_idx), max_evict, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev))
    if status is not None or sync:
        if status is not None and (not status.is_cuda or status.dtype != torch.int32):
            raise TypeError("status must be a CUDA int32 tensor")
        st = lib().dropkv_select_ex(*args, _ptr(status))
    else:
        st = lib().dropkv_select(*args)
    _check(st, "dropkv_select")
    return keep_idx, evict_idx


def dropkv_scores_select(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int,
                         pool_kernel: int, keep_counts: Sequence[int],
                         lengths: Optional[Sequence[int]] = None, *, path: str = "auto",
                         score: str = "perturbation", out: Optional[torch.Tensor] = None,
                         keep_idx: Optional[torch.Tensor] = None,
                         evict_idx: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, kernel_events=None,
                         tc_ctas: int = 0):
    """Scores and the keep / evict lists in one call (dropkv_scores_select):
    (scores, keep_idx, evict_idx), the same results as dropkv_scores followed
    by dropkv_select.  With ``status`` the call is asynchronous (the device
    status lands there); otherwise it synchronises and raises on a
    device-side error.  ``kernel_events`` as for dropkv_scores."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    _check_inputs(q, k, v)
    shape = make_shape(q, k, window, pool_kernel)
    dev = q.device
    B, Hkv, n_max = shape.B, shape.Hkv, shape.n_max
    lens = list(lengths) if lengths is not None else [n_max] * B
    keep = [int(x) for x in keep_counts]
    if len(keep) != B or len(lens) != B:
        raise ValueError("keep_counts and lengths need one entry per batch row")
    max_keep = max(keep)
    max_evict = max(L - kc for L, kc in zip(lens, keep))
    if out is None:
        out = torch.empty(B, Hkv, n_max, dtype=torch.float32, device=dev)
    if keep_idx is None:
        keep_idx = torch.empty(B, Hkv, max_keep, dtype=torch.int32, device=dev)
    if evict_idx is None:
        evict_idx = torch.empty(B, Hkv, max_evict, dtype=torch.int32, device=dev)
    need = scores_workspace_bytes(shape)
    if need == 0:
        raise DropKVError(ERR_ARG, "dropkv_scores_workspace_bytes")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    opts = Options(_PATHS[path], _SCORES[score], None, None, None, 0, int(tc_ctas))
    ev_arr = None
    if kernel_events:
        ev_arr = (ctypes.c_void_p * len(kernel_events))(*[e.cuda_event for e in kernel_events])
        opts.events = ctypes.cast(ev_arr, ctypes.c_void_p)
        opts.n_events = len(kernel_events)
    if status is not None and (not status.is_cuda or status.dtype != torch.int32):
        raise TypeError("status must be a CUDA int32 tensor")
    st = lib().dropkv_scores_select(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                    _i32_array(lengths), _i32_array(keep), _ptr(out),
                                    _ptr(keep_idx), keep_idx.shape[2], _ptr(evict_idx),
                                    evict_idx.shape[2], _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(dev),
                                    _ptr(status), ctypes.byref(opts))
    _check(st, "dropkv_scores_select")
    return out, keep_idx, evict_idx


def evict(q, k, v, window: int, pool_kernel: int, keep_counts: Sequence[int],
          lengths: Optional[Sequence[int]] = None, *, path: str = "auto",
          score: str = "perturbation"):
    """Scores and the keep / evict lists in one call: (scores, keep_idx, evict_idx)."""
    return dropkv_scores_select(q, k, v, window, pool_kernel, keep_counts, lengths, path=path,
                                score=score)


# ---- paged cache -----------------------------------------------------------------


# The library's structs as bytes: a decoding step makes two of these calls per
# layer, and packing takes a fraction of the time of filling a ctypes.Structure
# (whose layouts these are).
_CACHE_BYTES = struct.Struct("8i5Q").pack
_ROWS_BYTES = struct.Struct("2Q6q4i3Q").pack
_ATTN_BYTES = struct.Struct("3Q6q4ifi2Q").pack


@functools.lru_cache(maxsize=None)
def _packed_calls():
    """The cache entry points with their structs as bytes: (write, read, attention,
    attention's workspace)."""
    L, b, vp, sz = lib(), ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t
    out = []
    for name, args, res in (("dropkv_cache_write", [b, b, vp, vp], ctypes.c_int32),
                            ("dropkv_cache_read", [b, b, vp, vp], ctypes.c_int32),
                            ("dropkv_cache_attention", [b, b, vp, sz, vp, vp], ctypes.c_int32),
                            ("dropkv_cache_attention_workspace_bytes", [b, b], sz)):
        fn = L[name]  # an object of its own: the prototypes above stay
        fn.argtypes, fn.restype = args, res
        out.append(fn)
    return tuple(out)


def _cache(k_pages, v_pages, page_table, k_scale, v_scale) -> bytes:
    """Checks the pages' tensors and describes them to the library."""
    if not (isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor)
            and k_pages.is_cuda and v_pages.is_cuda):
        raise TypeError("k_pages and v_pages must be CUDA tensors (there is no CPU path)")
    shape, dev, dtype = k_pages.shape, k_pages.device, k_pages.dtype
    dt = _PAGE_DTYPES.get(dtype)
    if dt is None or v_pages.dtype not in _PAGE_DTYPES:
        raise TypeError("pages must be bfloat16, float32 or float8_e4m3fn")
    if len(shape) != 4 or not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise ValueError("pages must be contiguous [n_pages, Hkv, page_size, d] tensors")
    if v_pages.shape != shape or v_pages.dtype != dtype or v_pages.device != dev:
        raise ValueError("k_pages and v_pages must agree in shape, dtype and device")
    n_pages, Hkv, page_size, d = shape
    table = _int32_on(page_table, "page_table", dev)
    if table is None or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    ks = vs = 0
    if dt == E4M3 or k_scale is not None or v_scale is not None:
        if dt != E4M3 or k_scale is None or v_scale is None:
            raise ValueError("e4m3 pages come with k_scale and v_scale, other pages without")
        rows = shape[:3]
        for t in (k_scale, v_scale):
            if t.dtype != torch.uint8 or t.device != dev or not t.is_contiguous():
                raise TypeError("scales must be contiguous uint8 tensors on the pages' device")
            if t.shape != rows:
                raise ValueError("scales must be [n_pages, Hkv, page_size]")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    B, max_pages = page_table.shape
    return _CACHE_BYTES(B, Hkv, d, n_pages, page_size, max_pages, dt, 0, k_pages.data_ptr(),
                        v_pages.data_ptr(), ks, vs, table)


def _rank(t) -> int:
    """Dimensions of a tensor, 0 of anything else."""
    return t.dim() if isinstance(t, torch.Tensor) else 0


def _int32_on(t, name, device, shape=None):
    """The address of an int32 tensor on the pages' device; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise TypeError(f"{name} must be an int32 tensor on the pages' device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {list(shape)}")
    return t.data_ptr()


def _dense(t, name, device, shape):
    """Strides of a dense bf16 / fp32 tensor whose last index is contiguous."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError(f"{name} must be a CUDA tensor on the pages' device")
    if t.dtype not in _DENSE_DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {list(shape)}")
    st = t.stride()
    if st[3] != 1 and shape[3] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return st[:3]


def _written(t, name):
    """A tensor that a call writes: no element may stand for two indices."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor on the pages' device")
    if t.is_contiguous():
        return
    last = 0  # offset of the last element over the strides so far
    for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1),
                               key=lambda x: x[1]):
        if stride <= last:
            raise ValueError(f"{name} must not overlap itself")
        last += stride * (size - 1)


def _launch(fn, what, args, device, status, sync):
    """Calls fn(*args, status word, stream) on the pages' device; with ``sync``,
    waits and checks the status."""
    if status is not None:
        if status.dtype != torch.int32 or status.device != device or status.numel() < 1:
            raise TypeError("status must be a CUDA int32 tensor on the pages' device")
    elif sync:
        status = torch.empty(1, dtype=torch.int32, device=device)
    word = None if status is None else status.data_ptr()
    if device.index == torch.cuda.current_device():
        code = fn(*args, word, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, word, _raw_stream(device.index))
    if code != OK:
        _check(code, what)
    if sync:
        torch.cuda.current_stream(device).synchronize()
        _check(int(status.view(-1)[0].item()), what)


def _move(fn, what, dense, pages, n, rows, start, counts, status, sync):
    k, v = dense
    c = _cache(*pages)
    k_pages, _, page_table, _, _ = pages
    dev = k_pages.device
    B, shape = page_table.shape[0], k_pages.shape
    Hkv = shape[1]
    dense_shape = (B, Hkv, n, shape[3])
    ks, vs = _dense(k, "k", dev, dense_shape), _dense(v, "v", dev, dense_shape)
    if k.dtype != v.dtype:
        raise TypeError("k and v must share one dtype")
    m = n if rows is None else rows.shape[-1] if _rank(rows) else 0
    r = (None if rows is None else _int32_on(rows, "rows", dev, (B, Hkv, m)),
         None if start is None else _int32_on(start, "start", dev, (B,)),
         None if counts is None else _int32_on(counts, "counts", dev, (B,)))
    if m == 0 or n == 0:  # nothing to move
        if status is not None:
            status.zero_()
        return
    r = _ROWS_BYTES(k.data_ptr(), v.data_ptr(), *ks, *vs, _DENSE_DTYPES[k.dtype], n, m, 0,
                    r[0] or 0, r[1] or 0, r[2] or 0)
    _launch(fn, what, (c, r), dev, status, sync)


def dropkv_cache_write(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                       v_pages: torch.Tensor, page_table: torch.Tensor, *,
                       rows: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                       counts: Optional[torch.Tensor] = None,
                       k_scale: Optional[torch.Tensor] = None,
                       v_scale: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, sync: bool = False) -> None:
    """Writes dense K/V rows into a paged cache (dropkv_cache_write).

    k, v: [B, Hkv, n, d], bf16 or fp32, any strides with a contiguous last
    dimension (a transposed [B, n, Hkv, d] is fine).  k_pages, v_pages:
    [n_pages, Hkv, page_size, d] in bf16, fp32 or float8_e4m3fn, the last with
    uint8 scales k_scale, v_scale [n_pages, Hkv, page_size] (2^(byte - 127) a
    row).  page_table: int32 [B, max_pages].
    Slot start[b] + i of sequence b receives row i, or row rows[b, h, i] of a
    list (int32 [B, Hkv, m], such as dropkv_select's keep_idx; -1 is skipped),
    for i < counts[b].  start and counts: int32 [B] on the device, None for 0
    and for all rows.
    Asynchronous.  With ``status`` (a CUDA int32 tensor of one element) the
    device-side status lands there (ERR_ARG: some page, slot, row or count was
    out of range; what it named was left out); ``sync=True`` waits and raises.
    """
    if _rank(k) != 4:
        raise ValueError("k must be a [B, Hkv, n, d] tensor")
    _move(_packed_calls()[0], "dropkv_cache_write", (k, v),
          (k_pages, v_pages, page_table, k_scale, v_scale), k.shape[2], rows, start, counts,
          status, sync)


def dropkv_cache_read(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                      n: int, *, rows: Optional[torch.Tensor] = None,
                      start: Optional[torch.Tensor] = None,
                      counts: Optional[torch.Tensor] = None,
                      k_scale: Optional[torch.Tensor] = None,
                      v_scale: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                      out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                      status: Optional[torch.Tensor] = None, sync: bool = False):
    """Dense (k, v) [B, Hkv, n, d] of a paged cache (dropkv_cache_read).

    Row i is slot start[b] + i of sequence b, or slot start[b] + rows[b, h, i]
    of a list (int32 [B, Hkv, n]; -1 is skipped), for i < counts[b].  Rows that
    are not written keep ``out``'s values, or are 0 without ``out``.  ``dtype``:
    bf16 or fp32 (default: the pages' own, bf16 for e4m3 pages).  The other
    arguments are dropkv_cache_write's.
    """
    if rows is not None and (_rank(rows) != 3 or rows.shape[-1] != n):
        raise ValueError("rows must be an int32 tensor that lists n slots per (sequence, head)")
    if n < 0:
        raise ValueError("n must not be negative")
    if out is None:
        if _rank(k_pages) != 4 or _rank(page_table) != 2:
            raise ValueError("pages must be [n_pages, Hkv, page_size, d] tensors, page_table [B, max_pages]")
        dtype = dtype or (k_pages.dtype if k_pages.dtype in _DENSE_DTYPES else torch.bfloat16)
        shape = (page_table.shape[0], k_pages.shape[1], n, k_pages.shape[3])
        out = tuple(torch.zeros(shape, dtype=dtype, device=k_pages.device) for _ in range(2))
    else:
        for name, t in zip(("k", "v"), out):
            _written(t, f"out {name}")
            if dtype is not None and t.dtype != dtype:
                raise TypeError("out and dtype disagree")
    _move(_packed_calls()[1], "dropkv_cache_read", out,
          (k_pages, v_pages, page_table, k_scale, v_scale), n, rows, start, counts, status, sync)
    return out


def cache_attention_workspace_bytes(cache: Cache, attn: CacheAttn) -> int:
    return int(lib().dropkv_cache_attention_workspace_bytes(ctypes.byref(cache),
                                                            ctypes.byref(attn)))


def cache_attention_workspace(q: torch.Tensor, k_pages: torch.Tensor, page_table: torch.Tensor, *,
                              path: str = "auto") -> torch.Tensor:
    """A workspace for dropkv_cache_attention calls of q's and the pages' shapes and
    dtypes (lengths and values do not matter), on the pages' device: what a captured
    graph, or a loop of calls on one stream, passes as ``workspace=``."""
    (B, Hq, T, d), (n_pages, Hkv, page_size, page_d) = q.shape, k_pages.shape
    if k_pages.dtype not in _PAGE_DTYPES or q.dtype not in _DENSE_DTYPES:
        raise TypeError("q must be bfloat16 or float32, pages those or float8_e4m3fn")
    if d != page_d or B != page_table.shape[0]:
        raise ValueError("q must be [B, Hq, T, d] with the pages' B and d")
    if T == 0:  # no rows, no work
        return torch.empty(0, dtype=torch.uint8, device=k_pages.device)
    c = _CACHE_BYTES(B, Hkv, d, n_pages, page_size, page_table.shape[1],
                     _PAGE_DTYPES[k_pages.dtype], 0, 0, 0, 0, 0, 0)
    a = _ATTN_BYTES(0, 0, 0, *[0] * 6, _DENSE_DTYPES[q.dtype], Hq, T, 1, 0.0, _PATHS[path], 0, 0)
    need = _packed_calls()[3](c, a)
    if need == 0:
        raise DropKVError(ERR_ARG, "dropkv_cache_attention_workspace_bytes")
    return torch.empty(need, dtype=torch.uint8, device=k_pages.device)


def cache_attention_path(cache: Cache, attn: CacheAttn) -> int:
    return int(lib().dropkv_cache_attention_path(ctypes.byref(cache), ctypes.byref(attn)))


def dropkv_cache_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                           page_table: torch.Tensor, lengths: torch.Tensor, *,
                           q_lengths: Optional[torch.Tensor] = None,
                           scale: Optional[float] = None, causal: bool = True,
                           k_scale: Optional[torch.Tensor] = None,
                           v_scale: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           return_lse: bool = False, path: str = "auto",
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, sync: bool = False):
    """Attention of a chunk of new tokens over a paged cache
    (dropkv_cache_attention): out [B, Hq, T, d], or (out, lse).

    q: [B, Hq, T, d], bf16 or fp32, any strides with a contiguous last
    dimension.  lengths: int32 [B] on the device, the slots of each sequence
    with the chunk's own tokens (written beforehand) as the last ones.
    q_lengths: int32 [B], the tokens of each chunk (None: T); rows behind them
    keep ``out``'s and ``lse``'s values (0 without ``out`` / ``lse``).  Row t
    sees the slots up to its own position, all of them with ``causal=False``.
    A row that sees nothing gives 0 and a log-sum-exp of -inf.  ``scale``:
    default 1/sqrt(d).  ``lse``: fp32 [B, Hq, T], natural logarithm; returned
    with ``return_lse`` or when given.  ``path``: "auto", "simt" (fp32 CUDA
    cores) or "tensor".  ``workspace``: a tensor of cache_attention_workspace's
    (one that is too small, or None, is replaced by an allocation); calls that
    overlap need one each.  The other arguments are dropkv_cache_write's.
    """
    # in fp32, where a small one would become the library's 0 for the default
    if scale is not None and not 0.0 < ctypes.c_float(scale).value < float("inf"):
        raise ValueError("scale must be positive and finite in fp32")
    c = _cache(k_pages, v_pages, page_table, k_scale, v_scale)
    dev = k_pages.device
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B, Hq, T, d]")
    shape = q.shape
    B, Hq, T, d = shape
    _, Hkv, _, page_d = k_pages.shape
    if B != page_table.shape[0] or d != page_d or Hkv < 1 or Hq % Hkv:
        raise ValueError("q must be [B, Hq, T, d] with the pages' B and d and Hq a multiple of Hkv")
    qs = _dense(q, "q", dev, shape)
    if out is None:
        out = torch.zeros(shape, dtype=q.dtype, device=dev) if q_lengths is not None else \
            torch.empty(shape, dtype=q.dtype, device=dev)
    os_ = _dense(out, "out", dev, shape)
    _written(out, "out")
    if out.dtype != q.dtype:
        raise TypeError("out must have q's dtype")
    if lse is not None:
        if lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous() \
                or lse.shape != (B, Hq, T):
            raise ValueError("lse must be a contiguous fp32 [B, Hq, T] tensor on the pages' device")
        return_lse = True
    elif return_lse:
        lse = torch.zeros(B, Hq, T, device=dev)
    if lengths is None:
        raise ValueError("lengths are needed")
    a = _ATTN_BYTES(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), *qs, *os_,
                    _DENSE_DTYPES[q.dtype], Hq, T, 1 if causal else 0, scale or 0.0, _PATHS[path],
                    _int32_on(lengths, "lengths", dev, (B,)),
                    0 if q_lengths is None else _int32_on(q_lengths, "q_lengths", dev, (B,)))
    if T == 0:  # no rows
        if status is not None:
            status.zero_()
        return (out, lse) if return_lse else out
    _, _, attend, workspace_bytes = _packed_calls()
    need = workspace_bytes(c, a)
    if need == 0:
        raise DropKVError(ERR_ARG, "dropkv_cache_attention_workspace_bytes")
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != dev \
                or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous tensor on the pages' device")
        size = workspace.numel() * workspace.element_size()
    if workspace is None or size < need:
        workspace, size = torch.empty(need, dtype=torch.uint8, device=dev), need
    _launch(attend, "dropkv_cache_attention", (c, a, workspace.data_ptr(), size), dev, status, sync)
    return (out, lse) if return_lse else out


def selftest_cache_attention_timeout(T: int = 40, e4m3: bool = False, d: int = 128, B: int = 2,
                                     limit_ms: float = 20.0, device=None) -> int:
    """Runs dropkv_cache_attention's tcgen05 kernel over a small cache (B sequences
    of some 400 slots, two query heads on one KV head, T > 8 new tokens) with one
    hand-over of every CTA withheld and its waits limited to ``limit_ms``; returns the
    status word: ERR_TIMEOUT when they gave up as designed."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else \
        torch.device(device)
    pages = 16  # the sequences share them
    table = torch.arange(pages, dtype=torch.int32, device=dev).repeat(B, 1)
    q = torch.zeros(B, 2, T, d, dtype=torch.bfloat16, device=dev)
    out = torch.empty_like(q)
    lengths = torch.tensor([400 + b % 12 for b in range(B)], dtype=torch.int32, device=dev)
    kv = torch.zeros(pages, 1, 32, d, dtype=torch.uint8 if e4m3 else torch.bfloat16, device=dev)
    scale = torch.zeros(pages, 1, 32, dtype=torch.uint8, device=dev)
    strides = (ctypes.c_int64 * 3)(*q.stride()[:3])
    c = Cache(B, 1, d, pages, 32, pages, E4M3 if e4m3 else BF16, 0, kv.data_ptr(), kv.data_ptr(),
              scale.data_ptr() if e4m3 else None, scale.data_ptr() if e4m3 else None,
              table.data_ptr())
    a = CacheAttn(q.data_ptr(), out.data_ptr(), None, strides, strides, BF16, 2, T, 1, 0.0,
                  PATH_TENSOR, lengths.data_ptr(), None)
    size = cache_attention_workspace_bytes(c, a)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().dropkv_selftest_cache_attention_timeout(
            ctypes.byref(c), ctypes.byref(a), _ptr(ws), size, _ptr(status), int(limit_ms * 1e6),
            _stream(dev)), "dropkv_selftest_cache_attention_timeout")
    torch.cuda.synchronize(dev)
    return int(status.item())


def evict_to_cache(q, k, v, window: int, pool_kernel: int, keep_counts: Sequence[int],
                   k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                   lengths: Optional[Sequence[int]] = None, *,
                   k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, path: str = "auto",
                   score: str = "perturbation"):
    """Scores the prompt's tokens, lists the kept ones, and writes their K/V rows
    into slots 0.. of a paged cache: (cache lengths int32 [B], scores, keep_idx,
    evict_idx).  The arguments are evict's and dropkv_cache_write's, and refused
    before any work."""
    _cache(k_pages, v_pages, page_table, k_scale, v_scale)
    dev, (_, Hkv, _, d) = k_pages.device, k_pages.shape
    _check_inputs(q, k, v)
    shape = (page_table.shape[0], Hkv, k.shape[2] if k.dim() == 4 else 0, d)
    _dense(k, "k", dev, shape), _dense(v, "v", dev, shape)
    keep = [int(x) for x in keep_counts]
    if keep and max(keep) > page_table.shape[1] * k_pages.shape[2]:
        raise ValueError("the page table has too few pages for the kept tokens")
    scores, keep_idx, evict_idx = evict(q, k, v, window, pool_kernel, keep, lengths, path=path,
                                        score=score)
    counts = torch.tensor(keep, dtype=torch.int32, device=q.device)
    dropkv_cache_write(k, v, k_pages, v_pages, page_table, rows=keep_idx, counts=counts,
                       k_scale=k_scale, v_scale=v_scale, sync=True)
    return counts, scores, keep_idx, evict_idx
