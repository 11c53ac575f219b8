"""Python binding of libfd.so: single-token split-KV decode attention
(Flash-Decoding) over a position-addressed bf16 or FP8 (E4M3) KV cache on GB300.

Every function here has the name of the C entry point it wraps
(include/fd_decode_attn.h) and only marshals arguments: torch tensors become
device pointers, the current torch stream becomes the CUDA stream, non-zero
status codes become FdError. All arithmetic runs in libfd.so's kernels. There
is no fallback: if libfd.so is missing or a call fails, an exception is raised.
Where Python headers were available at build time, fd_decode_attn,
fd_decode_attn_fp8 and the calls of the paged cache go through the small
compiled module _fdfast (the same libfd.so, less host time per call);
elsewhere they go through ctypes.

Typical use in a decode loop (every layer its own cache; lens counts the
current token, whose K/V are already in the cache):

    import torch, decode_attention_04_gb300 as fd
    # q: bf16 [B, NH, HS]; k, v: bf16 [B, NKV, capacity, HS]; lens: int32 [B]
    out = fd.decode_attention(q, k, v, lens, window=1024)      # allocates out
    fd.fd_decode_attn(q, k, v, out, lens, B, NH, NKV, HS, capacity, window,
                      0.0)                                      # into out

The first call for a (device, stream) sizes the library's workspace; later
calls may be captured in a CUDA graph. fd_plan / fd_decode_attn_ex take an
explicit plan and workspace instead (nothing allocated by the library), and
fd_decode_attn_noalloc uses a fixed scratch array compiled into libfd.so.

With a cache in pages (include/fd_paged_attn.h), one decode step of all layers:

    # k_pages, v_pages: [layers, num_pages, NKV, page_size, HS] bf16, or uint8 E4M3 codes with
    # k_scale, v_scale: fp32 [layers, num_pages, NKV]; table int32 [B, max_pages], lens [B], refs [num_pages]
    fd.fd_pages_reserve(table, lens, refs, None, granted, moves, ws, ws.numel(), B, max_pages, num_pages, page_size)
    fd.fd_pages_copy(k_pages, v_pages, k_scale, v_scale, moves, B, layers, num_pages, NKV, page_size, HS, fd.FD_KV_E4M3)
    for n in range(layers):
        # k, v: the layer's new tokens [B, NKV, HS] bf16
        fd.fd_paged_append(k, v, k_pages[n], v_pages[n], k_scale[n], v_scale[n], table, lens, None, granted, B, B, NKV,
                           HS, page_size, num_pages, max_pages, k.stride(0), v.stride(0), fd.FD_KV_E4M3)
        out = fd.paged_attention(q, k_pages[n], v_pages[n], table, lens, k_scale=k_scale[n], v_scale=v_scale[n])
"""

from __future__ import annotations

import ctypes
from pathlib import Path

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libfd.so"

FD_OK = 0
FD_ERR_INVALID_ARG = 1
FD_ERR_UNSUPPORTED = 2
FD_ERR_ALIGNMENT = 3
FD_ERR_CUDA = 4
FD_ERR_WORKSPACE = 5
FD_ERR_SCRATCH_LIMIT = 6
FD_NOALLOC_SCRATCH_BYTES = 32 << 20

FD_DEVERR_LEN_NEGATIVE = 1 << 0
FD_DEVERR_LEN_CLAMPED = 1 << 1
FD_DEVERR_WAIT_TIMEOUT = 1 << 2
FD_DEVERR_MIN_LEN = 1 << 3
FD_DEVERR_PAGE_ID = 1 << 4
FD_DEVERR_PAGES_EXHAUSTED = 1 << 5

FD_PATH_AUTO = 0
FD_PATH_SIMT = 1
FD_PATH_TC = 2
FD_PATH_UMMA = 3

FD_KV_BF16 = 0
FD_KV_E4M3 = 1

EXPORTED = ["fd_plan", "fd_plan_sms", "fd_plan_kv", "fd_plan_sms_kv", "fd_plan_override", "fd_plan_persistent",
            "fd_plan_min_len", "fd_workspace_bytes",
            "fd_decode_attn", "fd_decode_attn_ex", "fd_decode_attn_fp8", "fd_decode_attn_fp8_ex",
            "fd_decode_attn_noalloc", "fd_debug_withhold_copies", "fd_get_device_error", "fd_release",
            "fd_strerror", "fd_version",
            "fd_paged_plan", "fd_paged_plan_sms", "fd_paged_attn", "fd_paged_attn_ex", "fd_paged_append",
            "fd_pages_workspace_bytes", "fd_pages_reserve", "fd_pages_fork", "fd_pages_free", "fd_pages_compact",
            "fd_pages_copy"]


class fd_plan_t(ctypes.Structure):
    _fields_ = [
        ("num_splits", ctypes.c_int),
        ("path", ctypes.c_int),
        ("cluster", ctypes.c_int),
        ("granule", ctypes.c_int),
        ("max_band", ctypes.c_int),
        ("ctas_per_sm", ctypes.c_int),
        ("num_sms", ctypes.c_int),
        ("max_cluster", ctypes.c_int),
        ("fused", ctypes.c_int),
        ("group_bytes", ctypes.c_int),
        ("kv_dtype", ctypes.c_int),
        ("consumer_warps", ctypes.c_int),
        ("persistent", ctypes.c_int),
        ("min_len", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
        ("workspace_zero_bytes", ctypes.c_size_t),
        ("B", ctypes.c_int),
        ("NH", ctypes.c_int),
        ("NKV", ctypes.c_int),
        ("HS", ctypes.c_int),
        ("capacity", ctypes.c_int),
        ("window", ctypes.c_int),
    ]

    def __repr__(self):
        return "fd_plan_t(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class fd_paged_plan_t(ctypes.Structure):
    _fields_ = [
        ("blocks", ctypes.c_int),
        ("granule", ctypes.c_int),
        ("min_share", ctypes.c_int),
        ("num_sms", ctypes.c_int),
        ("kv_dtype", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
        ("B", ctypes.c_int),
        ("NH", ctypes.c_int),
        ("NKV", ctypes.c_int),
        ("HS", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("max_pages", ctypes.c_int),
        ("window", ctypes.c_int),
    ]

    def __repr__(self):
        return "fd_paged_plan_t(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class FdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fd_strerror(status)} (status {status})")


_lib = None


def load_library(path: Path | str | None = None):
    """Load libfd.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    p = Path(path) if path else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build the CUDA library first "
                           "(python -m decode_attention_04_gb300.build)")
    lib = ctypes.CDLL(str(p))
    ci, vp, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    planp, ppagedp, ll = ctypes.POINTER(fd_plan_t), ctypes.POINTER(fd_paged_plan_t), ctypes.c_longlong
    sig = {
        "fd_plan": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, planp]),
        "fd_plan_sms": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, planp]),
        "fd_plan_kv": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, ci, planp]),
        "fd_plan_sms_kv": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, planp]),
        "fd_plan_override": (ci, [planp, ci, ci, ci, ci]),
        "fd_plan_persistent": (ci, [planp, ci]),
        "fd_plan_min_len": (ci, [planp, ci]),
        "fd_debug_withhold_copies": (ci, [ci, ctypes.c_ulonglong]),
        "fd_workspace_bytes": (sz, [planp]),
        "fd_decode_attn": (ci, [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ctypes.c_float, vp]),
        "fd_decode_attn_ex": (ci, [planp, vp, sz, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci,
                                   ctypes.c_float, vp]),
        "fd_decode_attn_fp8": (ci, [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ctypes.c_float, vp]),
        "fd_decode_attn_fp8_ex": (ci, [planp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci,
                                       ctypes.c_float, vp]),
        "fd_decode_attn_noalloc": (ci, [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ctypes.c_float, vp]),
        "fd_get_device_error": (ci, [vp, ctypes.POINTER(ctypes.c_uint)]),
        "fd_release": (None, []),
        "fd_strerror": (ctypes.c_char_p, [ci]),
        "fd_version": (ci, []),
        "fd_paged_plan": (ci, [ci] * 9 + [ppagedp]),
        "fd_paged_plan_sms": (ci, [ci] * 9 + [ppagedp]),
        "fd_paged_attn": (ci, [vp] * 8 + [ci] * 8 + [ctypes.c_float, ci, vp]),
        "fd_paged_attn_ex": (ci, [ppagedp, vp, sz] + [vp] * 9 + [ci] * 8 + [ctypes.c_float, vp]),
        "fd_paged_append": (ci, [vp] * 10 + [ci] * 7 + [ll, ll, ci, vp]),
        "fd_pages_workspace_bytes": (sz, [ci, ci]),
        "fd_pages_reserve": (ci, [vp] * 7 + [sz] + [ci] * 4 + [vp]),
        "fd_pages_fork": (ci, [vp] * 6 + [ci] * 4 + [vp]),
        "fd_pages_free": (ci, [vp] * 4 + [ci] * 5 + [vp]),
        "fd_pages_compact": (ci, [vp] * 4 + [sz] + [ci] * 3 + [vp]),
        "fd_pages_copy": (ci, [vp] * 5 + [ci] * 7 + [vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != FD_OK:
        raise FdError(rc, where)


def fd_strerror(status: int) -> str:
    return load_library().fd_strerror(status).decode()


def fd_version() -> int:
    return load_library().fd_version()


def fd_plan(B, NH, NKV, HS, capacity, window, max_len=0, device=None) -> fd_plan_t:
    if device is None:
        import torch
        device = torch.cuda.current_device()
    p = fd_plan_t()
    _check(load_library().fd_plan(B, NH, NKV, HS, capacity, window, max_len, int(device), ctypes.byref(p)),
           "fd_plan")
    return p


def fd_plan_sms(B, NH, NKV, HS, capacity, window, max_len, num_sms, ctas_per_sm, max_cluster=8) -> fd_plan_t:
    p = fd_plan_t()
    _check(load_library().fd_plan_sms(B, NH, NKV, HS, capacity, window, max_len, num_sms, ctas_per_sm,
                                      max_cluster, ctypes.byref(p)), "fd_plan_sms")
    return p


def fd_plan_kv(B, NH, NKV, HS, capacity, window, max_len=0, device=None, kv_dtype=FD_KV_BF16) -> fd_plan_t:
    if device is None:
        import torch
        device = torch.cuda.current_device()
    p = fd_plan_t()
    _check(load_library().fd_plan_kv(B, NH, NKV, HS, capacity, window, max_len, int(device), int(kv_dtype),
                                     ctypes.byref(p)), "fd_plan_kv")
    return p


def fd_plan_sms_kv(B, NH, NKV, HS, capacity, window, max_len, num_sms, ctas_per_sm, max_cluster=8,
                   kv_dtype=FD_KV_BF16) -> fd_plan_t:
    p = fd_plan_t()
    _check(load_library().fd_plan_sms_kv(B, NH, NKV, HS, capacity, window, max_len, num_sms, ctas_per_sm,
                                         max_cluster, int(kv_dtype), ctypes.byref(p)), "fd_plan_sms_kv")
    return p


def fd_plan_override(plan: fd_plan_t, num_splits: int = 0, path: int = FD_PATH_AUTO, cluster: int = 0,
                     fused: int = -1) -> fd_plan_t:
    _check(load_library().fd_plan_override(ctypes.byref(plan), num_splits, path, cluster, fused),
           "fd_plan_override")
    return plan


def fd_plan_persistent(plan: fd_plan_t, persistent: int = 1) -> fd_plan_t:
    _check(load_library().fd_plan_persistent(ctypes.byref(plan), persistent), "fd_plan_persistent")
    return plan


def fd_plan_min_len(plan: fd_plan_t, min_len: int) -> fd_plan_t:
    """Record the caller's lower bound on every len_b (tiles of slots that any
    such length makes live may then be read before the lengths arrive)."""
    _check(load_library().fd_plan_min_len(ctypes.byref(plan), int(min_len)), "fd_plan_min_len")
    return plan


def fd_debug_withhold_copies(withhold_tile: int, wait_limit_ns: int = 0) -> None:
    """Test hook of the bounded waits: split blocks issue no copies from
    their tile `withhold_tile` on (< 0: off), and waits give up after
    `wait_limit_ns` (0: the default, about one second)."""
    _check(load_library().fd_debug_withhold_copies(int(withhold_tile), int(wait_limit_ns)),
           "fd_debug_withhold_copies")


def fd_workspace_bytes(plan: fd_plan_t) -> int:
    return load_library().fd_workspace_bytes(ctypes.byref(plan))


_fast_mod = None
_fast_for = None  # the ctypes handle the compiled entries belong to


def _fast():
    """The compiled CPython entries (``_fdfast``, linked to the in-tree
    libfd.so) when they were built and that library is the one loaded; else
    None, and calls go through ctypes."""
    global _fast_mod, _fast_for
    if _fast_for is not None and _fast_for is _lib:
        return _fast_mod
    lib = load_library()
    if _fast_for is not lib:
        _fast_for, _fast_mod = lib, None
        if Path(getattr(lib, "_name", "")).resolve() == LIB_PATH.resolve():
            try:
                from . import _fdfast
                _fast_mod = _fdfast
            except ImportError:
                _fast_mod = None
    return _fast_mod


def fd_decode_attn(q, k_cache, v_cache, out, lens, B, NH, NKV, HS, capacity, window, scale,
                   stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.decode_attn(_ptr(q) or 0, _ptr(k_cache) or 0, _ptr(v_cache) or 0, _ptr(out) or 0, _ptr(lens) or 0,
                           B, NH, NKV, HS, capacity, window, float(scale), _stream(stream) or 0)
    else:
        rc = load_library().fd_decode_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lens),
                                           B, NH, NKV, HS, capacity, window, float(scale), _stream(stream))
    _check(rc, "fd_decode_attn")


def fd_decode_attn_ex(plan: fd_plan_t, workspace, workspace_bytes, out_f32, q, k_cache, v_cache, out, lens,
                      B, NH, NKV, HS, capacity, window, scale, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.decode_attn_ex(ctypes.addressof(plan), _ptr(workspace) or 0, int(workspace_bytes), _ptr(out_f32) or 0,
                              _ptr(q) or 0, _ptr(k_cache) or 0, _ptr(v_cache) or 0, _ptr(out) or 0, _ptr(lens) or 0,
                              B, NH, NKV, HS, capacity, window, float(scale), _stream(stream) or 0)
    else:
        rc = load_library().fd_decode_attn_ex(ctypes.byref(plan), _ptr(workspace), int(workspace_bytes),
                                              _ptr(out_f32), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                              _ptr(lens), B, NH, NKV, HS, capacity, window, float(scale),
                                              _stream(stream))
    _check(rc, "fd_decode_attn_ex")


def fd_decode_attn_fp8(q, k8, v8, k_scale, v_scale, out, lens, B, NH, NKV, HS, capacity, window, scale,
                       stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.decode_attn_fp8(_ptr(q) or 0, _ptr(k8) or 0, _ptr(v8) or 0, _ptr(k_scale) or 0, _ptr(v_scale) or 0,
                               _ptr(out) or 0, _ptr(lens) or 0, B, NH, NKV, HS, capacity, window, float(scale),
                               _stream(stream) or 0)
    else:
        rc = load_library().fd_decode_attn_fp8(_ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale), _ptr(v_scale), _ptr(out),
                                               _ptr(lens), B, NH, NKV, HS, capacity, window, float(scale),
                                               _stream(stream))
    _check(rc, "fd_decode_attn_fp8")


def fd_decode_attn_fp8_ex(plan: fd_plan_t, workspace, workspace_bytes, out_f32, q, k8, v8, k_scale, v_scale, out,
                          lens, B, NH, NKV, HS, capacity, window, scale, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.decode_attn_fp8_ex(ctypes.addressof(plan), _ptr(workspace) or 0, int(workspace_bytes),
                                  _ptr(out_f32) or 0, _ptr(q) or 0, _ptr(k8) or 0, _ptr(v8) or 0, _ptr(k_scale) or 0,
                                  _ptr(v_scale) or 0, _ptr(out) or 0, _ptr(lens) or 0, B, NH, NKV, HS, capacity,
                                  window, float(scale), _stream(stream) or 0)
    else:
        rc = load_library().fd_decode_attn_fp8_ex(ctypes.byref(plan), _ptr(workspace), int(workspace_bytes),
                                                  _ptr(out_f32), _ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale),
                                                  _ptr(v_scale), _ptr(out), _ptr(lens), B, NH, NKV, HS, capacity,
                                                  window, float(scale), _stream(stream))
    _check(rc, "fd_decode_attn_fp8_ex")


def fd_decode_attn_noalloc(q, k_cache, v_cache, out, lens, B, NH, NKV, HS, capacity, window, scale,
                           stream=None) -> None:
    """fd_decode_attn for callers that must not allocate device memory while
    they run: the split partials go to a fixed 32 MiB array inside libfd.so.
    Calls that overlap on the GPU share that array and race; serialise them."""
    _check(load_library().fd_decode_attn_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lens),
                                                 B, NH, NKV, HS, capacity, window, float(scale),
                                                 _stream(stream)),
           "fd_decode_attn_noalloc")


def fd_get_device_error(stream=None) -> int:
    err = ctypes.c_uint(0)
    _check(load_library().fd_get_device_error(_stream(stream), ctypes.byref(err)), "fd_get_device_error")
    return err.value


def fd_release() -> None:
    load_library().fd_release()


def decode_attention(q, k_cache, v_cache, lens, window=0, scale=0.0, out=None, stream=None):
    """Convenience form over torch tensors: q [B,NH,HS], caches [B,NKV,capacity,HS]
    (bf16, CUDA), lens int32 [B] (CUDA). Allocates `out` if not given and calls
    fd_decode_attn."""
    import torch
    B, NH, HS = q.shape
    _, NKV, capacity, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    fd_decode_attn(q, k_cache, v_cache, out, lens, B, NH, NKV, HS, capacity, window, scale, stream)
    return out


# ------------------------------------------------------- the cache in pages


_current_raw = None


def _raw_stream(stream) -> int:
    """As _stream; the current stream without an object made for it, where torch offers that."""
    global _current_raw
    if stream is not None:
        return _stream(stream) or 0
    if _current_raw is None:
        import torch
        torch.cuda.current_device()  # initialises CUDA
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        _current_raw = (lambda: raw(device())) if raw and device else (lambda: _stream(None) or 0)
    return _current_raw()



def fd_paged_plan(B, NH, NKV, HS, page_size, max_pages, window, device=None, kv_dtype=FD_KV_BF16) -> fd_paged_plan_t:
    if device is None:
        import torch
        device = torch.cuda.current_device()
    p = fd_paged_plan_t()
    _check(load_library().fd_paged_plan(B, NH, NKV, HS, page_size, max_pages, window, int(device), int(kv_dtype),
                                        ctypes.byref(p)), "fd_paged_plan")
    return p


def fd_paged_plan_sms(B, NH, NKV, HS, page_size, max_pages, window, num_sms, kv_dtype=FD_KV_BF16) -> fd_paged_plan_t:
    p = fd_paged_plan_t()
    _check(load_library().fd_paged_plan_sms(B, NH, NKV, HS, page_size, max_pages, window, int(num_sms), int(kv_dtype),
                                            ctypes.byref(p)), "fd_paged_plan_sms")
    return p


def fd_paged_attn(q, k_pages, v_pages, k_scale, v_scale, out, table, lens, B, NH, NKV, HS, page_size, num_pages,
                  max_pages, window, scale, kv_dtype, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.paged_attn(q, k_pages, v_pages, k_scale, v_scale, out, table, lens, B, NH, NKV, HS, page_size,
                          num_pages, max_pages, window, scale, kv_dtype, _raw_stream(stream))
    else:
        rc = load_library().fd_paged_attn(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
                                          _ptr(out), _ptr(table), _ptr(lens), B, NH, NKV, HS, page_size, num_pages,
                                          max_pages, window, scale, kv_dtype, _stream(stream))
    _check(rc, "fd_paged_attn")


def fd_paged_attn_ex(plan: fd_paged_plan_t, workspace, workspace_bytes, out_f32, q, k_pages, v_pages, k_scale, v_scale,
                     out, table, lens, B, NH, NKV, HS, page_size, num_pages, max_pages, window, scale,
                     stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.paged_attn_ex(ctypes.addressof(plan), workspace, workspace_bytes, out_f32, q, k_pages, v_pages, k_scale,
                             v_scale, out, table, lens, B, NH, NKV, HS, page_size, num_pages, max_pages, window, scale,
                             _raw_stream(stream))
    else:
        rc = load_library().fd_paged_attn_ex(ctypes.byref(plan), _ptr(workspace), workspace_bytes, _ptr(out_f32),
                                             _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
                                             _ptr(out), _ptr(table), _ptr(lens), B, NH, NKV, HS, page_size, num_pages,
                                             max_pages, window, scale, _stream(stream))
    _check(rc, "fd_paged_attn_ex")


def fd_paged_append(k_new, v_new, k_pages, v_pages, k_scale, v_scale, table, lens, start, count, B, T, NKV, HS,
                    page_size, num_pages, max_pages, k_stride, v_stride, kv_dtype, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.paged_append(k_new, v_new, k_pages, v_pages, k_scale, v_scale, table, lens, start, count, B, T, NKV,
                            HS, page_size, num_pages, max_pages, k_stride, v_stride, kv_dtype, _raw_stream(stream))
    else:
        rc = load_library().fd_paged_append(_ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale),
                                            _ptr(v_scale), _ptr(table), _ptr(lens), _ptr(start), _ptr(count), B, T,
                                            NKV, HS, page_size, num_pages, max_pages, k_stride, v_stride, kv_dtype,
                                            _stream(stream))
    _check(rc, "fd_paged_append")


def fd_pages_workspace_bytes(B, num_pages) -> int:
    return load_library().fd_pages_workspace_bytes(B, num_pages)


def fd_pages_reserve(table, lens, refs, grow, granted, moves, workspace, workspace_bytes, B, max_pages, num_pages,
                     page_size, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.pages_reserve(table, lens, refs, grow, granted, moves, workspace, workspace_bytes, B, max_pages,
                             num_pages, page_size, _raw_stream(stream))
    else:
        rc = load_library().fd_pages_reserve(_ptr(table), _ptr(lens), _ptr(refs), _ptr(grow), _ptr(granted),
                                             _ptr(moves), _ptr(workspace), workspace_bytes, B, max_pages, num_pages,
                                             page_size, _stream(stream))
    _check(rc, "fd_pages_reserve")


def fd_pages_fork(table, lens, parent, table_out, lens_out, refs, B, B_out, max_pages, num_pages, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.pages_fork(table, lens, parent, table_out, lens_out, refs, B, B_out, max_pages, num_pages,
                          _raw_stream(stream))
    else:
        rc = load_library().fd_pages_fork(_ptr(table), _ptr(lens), _ptr(parent), _ptr(table_out), _ptr(lens_out),
                                          _ptr(refs), B, B_out, max_pages, num_pages, _stream(stream))
    _check(rc, "fd_pages_fork")


def fd_pages_free(table, lens, refs, keep, window, B, max_pages, num_pages, page_size, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.pages_free(table, lens, refs, keep, window, B, max_pages, num_pages, page_size, _raw_stream(stream))
    else:
        rc = load_library().fd_pages_free(_ptr(table), _ptr(lens), _ptr(refs), _ptr(keep), window, B, max_pages,
                                          num_pages, page_size, _stream(stream))
    _check(rc, "fd_pages_free")


def fd_pages_compact(table, refs, moves, workspace, workspace_bytes, B, max_pages, num_pages, stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.pages_compact(table, refs, moves, workspace, workspace_bytes, B, max_pages, num_pages,
                             _raw_stream(stream))
    else:
        rc = load_library().fd_pages_compact(_ptr(table), _ptr(refs), _ptr(moves), _ptr(workspace), workspace_bytes,
                                             B, max_pages, num_pages, _stream(stream))
    _check(rc, "fd_pages_compact")


def fd_pages_copy(k_pages, v_pages, k_scale, v_scale, moves, room, layers, num_pages, NKV, page_size, HS, kv_dtype,
                  stream=None) -> None:
    f = _fast()
    if f is not None:
        rc = f.pages_copy(k_pages, v_pages, k_scale, v_scale, moves, room, layers, num_pages, NKV, page_size, HS,
                          kv_dtype, _raw_stream(stream))
    else:
        rc = load_library().fd_pages_copy(_ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(moves),
                                          room, layers, num_pages, NKV, page_size, HS, kv_dtype, _stream(stream))
    _check(rc, "fd_pages_copy")


def paged_attention(q, k_pages, v_pages, table, lens, window=0, scale=0.0, k_scale=None, v_scale=None, out=None,
                    stream=None):
    """Convenience form over torch tensors: q [B,NH,HS] bf16, pages
    [num_pages,NKV,page_size,HS] (bf16, or E4M3 codes with k_scale and v_scale
    [num_pages,NKV] fp32), table int32 [B,max_pages], lens int32 [B], all
    contiguous on the current device. Allocates `out` if not given and calls
    fd_paged_attn."""
    import torch
    B, NH, HS = q.shape
    num_pages, NKV, page_size, _ = k_pages.shape
    if out is None:
        out = torch.empty_like(q)
    kv_dtype = FD_KV_BF16 if k_scale is None else FD_KV_E4M3
    _require(q=(q, torch.bfloat16, (B, NH, HS)), out=(out, torch.bfloat16, (B, NH, HS)),
             k_pages=(k_pages, _code_types() if kv_dtype else torch.bfloat16, (num_pages, NKV, page_size, HS)),
             v_pages=(v_pages, _code_types() if kv_dtype else torch.bfloat16, (num_pages, NKV, page_size, HS)),
             table=(table, torch.int32, (B, table.shape[-1])), lens=(lens, torch.int32, (B,)))
    if kv_dtype:
        _require(k_scale=(k_scale, torch.float32, (num_pages, NKV)), v_scale=(v_scale, torch.float32, (num_pages, NKV)))
    fd_paged_attn(q, k_pages, v_pages, k_scale, v_scale, out, table, lens, B, NH, NKV, HS, page_size, num_pages,
                  table.shape[1], window, scale, kv_dtype, stream)
    return out


def _code_types():
    import torch
    return (torch.uint8, torch.float8_e4m3fn)


def _require(**tensors):
    """The convenience forms hand bare addresses on: a tensor of another type,
    shape, layout or device is refused here."""
    import torch
    for name, (t, dtype, shape) in tensors.items():
        ok = (t is not None and t.is_cuda and t.device.index == torch.cuda.current_device() and t.is_contiguous() and
              tuple(t.shape) == tuple(shape))
        if not ok or t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
            raise FdError(FD_ERR_INVALID_ARG, f"{name}: contiguous tensor {tuple(shape)} of {dtype} on the current CUDA device expected")


__all__ = EXPORTED + ["fd_plan_t", "fd_paged_plan_t", "FdError", "load_library", "decode_attention", "paged_attention",
                      "LIB_PATH"]
