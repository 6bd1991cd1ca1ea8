"""ctypes binding of libfa_gb300.so -- argument marshalling only.

Every function here has the name of the C entry point it calls (declared in
include/fa.h).  Tensors are torch tensors used as device (or pinned host)
memory; all computation happens in the library's CUDA kernels.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "libfa_gb300.so")
_lib = None

FA_F16, FA_BF16 = 0, 1
FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED = 0, 1, 2
FA_ERR_CUDA, FA_ERR_WORKSPACE, FA_ERR_TIMEOUT = 3, 4, 5
FA_FLAG_NO_LPT = 0x1
FA_FLAG_ALWAYS_RESCALE = 0x2
FA_FLAG_EXACT_MAX = 0x4
FA_FLAG_PAIR = 0x8
FA_FLAG_SINGLE_CTA = 0x10
FA_FLAG_CORRECTION_WG = 0x20
FA_FLAG_PAIR64 = 0x40
FA_FLAG_OVERLAP_PREVIOUS = 0x80
FA_FLAG_TEST_STALL = 0x100
FA_FLAG_TAIL_SPLIT = 0x200
FA_FLAG_D64_THREE_STAGE = 0x400

_DTYPE = {torch.float16: FA_F16, torch.bfloat16: FA_BF16}


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {fa_status_string(status)} (status {status})")


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load the library; raises if it has not been built."""
    global _lib
    if _lib is None:
        _lib = load_path(_LIB_PATH)
    return _lib


def load_path(path: str) -> ctypes.CDLL:
    """Load a build of the library from ``path`` (the in-tree one, or
    another build of the same sources, e.g. a variant compared against it
    in a paired measurement).  Each build loads as its own module, with its
    own device state."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(path)
    vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    L.fa_fwd.restype = ci
    L.fa_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci]
    L.fa_workspace_bytes.restype = sz
    L.fa_fwd_ex.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci,
                            ctypes.c_uint, ci, vp, sz, vp]
    L.fa_fwd_ex.restype = ci
    L.fa_host_staging_bytes.argtypes = [ci, ci, ci, ci, ci]
    L.fa_host_staging_bytes.restype = sz
    L.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci,
                              ci, vp, sz, vp]
    L.fa_fwd_host.restype = ci
    L.fa_fwd_decode_static.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, cf,
                                       ci, vp]
    L.fa_fwd_decode_static.restype = ci
    L.fa_release_workspaces.argtypes = []
    L.fa_release_workspaces.restype = ci
    L.fa_get_device_status.argtypes = [vp]
    L.fa_get_device_status.restype = ci
    L.fa_set_watchdog_ns.argtypes = [ctypes.c_ulonglong]
    L.fa_set_watchdog_ns.restype = None
    L.fa_status_string.argtypes = [ci]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_prefill_uses_pairs.argtypes = [ci, ci, ci, ci, ci, ci, ctypes.c_uint, ci]
    L.fa_prefill_uses_pairs.restype = ci
    L.fa_ex2_approx.argtypes = [vp, vp, ci, vp]
    L.fa_ex2_approx.restype = ci
    L.fa_prefill_tail_items.argtypes = [ci, ci, ci, ci, ci, ci, ci, ctypes.c_uint]
    L.fa_prefill_tail_items.restype = ci
    L.fa_score_workspace_bytes.argtypes = [ci] * 7
    L.fa_score_workspace_bytes.restype = sz
    L.fa_fwd_score.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, cf,
                               vp, vp, vp, vp, vp, sz, vp]
    L.fa_fwd_score.restype = ci
    L.fa_cache_write.argtypes = [vp] * 9 + [ci] * 8 + [vp]
    L.fa_cache_write.restype = ci
    L.fa_cache_read.argtypes = [vp] * 9 + [ci] * 8 + [vp]
    L.fa_cache_read.restype = ci
    L.fa_cache_workspace_bytes.argtypes = [ci] * 8
    L.fa_cache_workspace_bytes.restype = sz
    L.fa_fwd_cache.argtypes = [vp] * 9 + [ci] * 9 + [cf, ci, cf, vp, vp, sz, vp]
    L.fa_fwd_cache.restype = ci
    L.fa_version.argtypes = []
    L.fa_version.restype = ci
    return L


def _stream_handle(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _shape(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, S, D]")
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if k.shape != (B, H, Skv, D) or v.shape != (B, H, Skv, D):
        raise ValueError("k and v must be [B, H, Skv, D] matching q")
    if q.dtype not in _DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype float16 or bfloat16")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    return B, H, Sq, Skv, D


def _outputs(q, out, lse):
    B, H, Sq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must match q")
    if lse.shape != (B, H, Sq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be float32 [B, H, Sq]")
    return out, lse


def _check(status: int, what: str) -> None:
    if status != FA_OK:
        raise FAError(status, what)


def fa_fwd(q, k, v, causal: bool = False, scale: float | None = None,
           out=None, lse=None, stream=None, lib=None):
    """O, LSE = attention(q, k, v) on the library's kernels.  Returns (o, lse).
    ``lib``: another loaded build (load_path); default the in-tree one."""
    B, H, Sq, Skv, D = _shape(q, k, v)
    out, lse = _outputs(q, out, lse)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    st = (lib or load()).fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                       lse.data_ptr(), B, H, Sq, Skv, D, sc, int(bool(causal)),
                       _DTYPE[q.dtype], _stream_handle(stream))
    _check(st, "fa_fwd")
    return out, lse


def fa_workspace_bytes(B: int, H: int, Sq: int, Skv: int, D: int,
                       num_splits: int = 0) -> int:
    return int(load().fa_workspace_bytes(B, H, Sq, Skv, D, num_splits))


def fa_fwd_ex(q, k, v, causal: bool = False, scale: float | None = None,
              flags: int = 0, num_splits: int = 0, workspace=None, out=None,
              lse=None, stream=None, lib=None):
    """fa_fwd with flags, an explicit decode split count and a caller-owned
    workspace tensor (any dtype, on the device)."""
    B, H, Sq, Skv, D = _shape(q, k, v)
    out, lse = _outputs(q, out, lse)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = workspace.data_ptr()
        ws_bytes = workspace.numel() * workspace.element_size()
    st = (lib or load()).fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                          out.data_ptr(), lse.data_ptr(), B, H, Sq, Skv, D, sc,
                          int(bool(causal)), _DTYPE[q.dtype], int(flags),
                          int(num_splits), ws_ptr, ws_bytes,
                          _stream_handle(stream))
    _check(st, "fa_fwd_ex")
    return out, lse


def fa_host_staging_bytes(B: int, H: int, Sq: int, Skv: int, D: int) -> int:
    return int(load().fa_host_staging_bytes(B, H, Sq, Skv, D))


def fa_fwd_host(q_h, k_h, v_h, staging, causal: bool = False,
                scale: float | None = None, out_h=None, lse_h=None,
                stream=None):
    """The forward pass on HOST tensors (pinned for full bandwidth): the
    library copies them into ``staging`` (a device tensor of at least
    fa_host_staging_bytes bytes), runs, and copies O and LSE back into
    ``out_h`` / ``lse_h`` (host).  Asynchronous on ``stream``."""
    B, H, Sq, Skv, D = _shape(q_h, k_h, v_h)
    if out_h is None:
        out_h = torch.empty_like(q_h, pin_memory=q_h.is_pinned())
    if lse_h is None:
        lse_h = torch.empty((B, H, Sq), dtype=torch.float32,
                            pin_memory=q_h.is_pinned())
    sc = float(D) ** -0.5 if scale is None else float(scale)
    st = load().fa_fwd_host(q_h.data_ptr(), k_h.data_ptr(), v_h.data_ptr(),
                            out_h.data_ptr(), lse_h.data_ptr(), B, H, Sq, Skv,
                            D, sc, int(bool(causal)), _DTYPE[q_h.dtype],
                            staging.data_ptr(),
                            staging.numel() * staging.element_size(),
                            _stream_handle(stream))
    _check(st, "fa_fwd_host")
    return out_h, lse_h


def fa_fwd_decode_static(q, k, v, scale: float | None = None, out=None,
                         lse=None, stream=None):
    """Decode (Sq == 1) without any device allocation: the split partials go
    to the library's static device scratch.  Calls whose GPU work overlaps
    share that scratch and race.  Returns (o, lse)."""
    B, H, Sq, Skv, D = _shape(q, k, v)
    if Sq != 1:
        raise ValueError("fa_fwd_decode_static takes one query row per head")
    out, lse = _outputs(q, out, lse)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    st = load().fa_fwd_decode_static(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     out.data_ptr(), lse.data_ptr(), B, H, Skv,
                                     D, sc, _DTYPE[q.dtype],
                                     _stream_handle(stream))
    _check(st, "fa_fwd_decode_static")
    return out, lse


class _Call:
    """The stream of a call on ``like``'s device, current for its length, and
    the memory that the call makes for itself there."""

    def __init__(self, like: torch.Tensor, stream):
        self.device, self.given = like.device, stream
        self.guard = torch.cuda.device(like.device)

    def __enter__(self):
        self.guard.__enter__()
        current = torch.cuda.current_stream()
        if self.given is None:
            self.handle, self.other = current.cuda_stream, None
        else:
            self.handle = _stream_handle(self.given)
            self.other = None
            if self.handle != current.cuda_stream:
                self.other = (self.given if isinstance(self.given, torch.cuda.Stream)
                              else torch.cuda.ExternalStream(self.handle, device=self.device))
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.other is not None:
            # made on the current stream: wait for the work that last had this
            # memory, and keep it until the call's own stream is done with it
            self.other.wait_stream(torch.cuda.current_stream())
            t.record_stream(self.other)
        return t

    def workspace(self, given, need: int):
        """(tensor, pointer, bytes) of the caller's workspace, or of one made
        for this call."""
        if given is None:
            given = self.empty((need,), torch.uint8) if need else None
        if given is None:
            return None, None, 0
        return given, given.data_ptr(), given.numel() * given.element_size()


def _cuda_tensor(t, name: str, like: torch.Tensor, dtype, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a tensor on q's (or k's) CUDA device")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _optional(t, name, like, dtype, shape):
    if t is None:
        return None
    _cuda_tensor(t, name, like, dtype, shape)
    return t.data_ptr()


def _rows16(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be a 4-d float16 or bfloat16 tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _grouped(q, Hkv: int):
    _rows16(q, "q")
    if Hkv < 1 or q.shape[1] % Hkv != 0:
        raise ValueError("the kv heads must divide the query heads")


def _given_outputs(call, q, out, lse):
    B, H, Sq, D = q.shape
    if out is None:
        out = call.empty(q.shape, q.dtype)
    if lse is None:
        lse = call.empty((B, H, Sq), torch.float32)
    _cuda_tensor(out, "out", q, q.dtype, q.shape)
    _cuda_tensor(lse, "lse", q, torch.float32, (B, H, Sq))
    return out, lse


def fa_score_workspace_bytes(B: int, H: int, Hkv: int, Sq: int, Skv: int, D: int,
                             documents: bool = False) -> int:
    return int(load().fa_score_workspace_bytes(B, H, Hkv, Sq, Skv, D, int(bool(documents))))


def fa_fwd_score(q, k, v, causal: bool = False, scale: float | None = None,
                 softcap: float = 0.0, slopes=None, doc_q=None, doc_k=None, prefix=None,
                 workspace=None, out=None, lse=None, stream=None):
    """Attention with modified scores on grouped heads: q [B, H, Sq, D], k and
    v [B, Hkv, Skv, D].  ``softcap`` caps the scores by a tanh, ``slopes``
    (float32 [H]) takes slope * distance off them, ``doc_q`` / ``doc_k``
    (int32 [B, Sq], [B, Skv]) keep rows to keys of their document, ``prefix``
    (int32 [B], causal only) shows the first keys to every row.  Without
    ``workspace`` the call makes its own.  Returns (o, lse)."""
    _rows16(k, "k")
    _grouped(q, k.shape[1])
    B, H, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    _cuda_tensor(k, "k", q, q.dtype, (B, Hkv, Skv, D))
    _cuda_tensor(v, "v", q, q.dtype, (B, Hkv, Skv, D))
    slopes_p = _optional(slopes, "slopes", q, torch.float32, (H,))
    doc_q_p = _optional(doc_q, "doc_q", q, torch.int32, (B, Sq))
    doc_k_p = _optional(doc_k, "doc_k", q, torch.int32, (B, Skv))
    prefix_p = _optional(prefix, "prefix", q, torch.int32, (B,))
    sc = float(D) ** -0.5 if scale is None else float(scale)
    with _Call(q, stream) as call:
        out, lse = _given_outputs(call, q, out, lse)
        need = 0
        if workspace is None:
            need = fa_score_workspace_bytes(B, H, Hkv, Sq, Skv, D, doc_k is not None)
        _keep, ws_ptr, ws_bytes = call.workspace(workspace, need)
        st = load().fa_fwd_score(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), B, H, Hkv, Sq, Skv, D, sc, int(bool(causal)),
                                 _DTYPE[q.dtype], float(softcap), slopes_p, doc_q_p, doc_k_p,
                                 prefix_p, ws_ptr, ws_bytes, call.handle)
    _check(st, "fa_fwd_score")
    return out, lse


def fa_cache_empty(num_pages: int, Hkv: int, page_size: int, D: int, device="cuda"):
    """The four arrays (k_codes, k_params, v_codes, v_params) of a 4-bit cache
    of that many pages, zeroed; any tensors of these shapes and types serve."""
    if D not in (64, 128):
        raise ValueError("D must be 64 or 128")
    rows = (num_pages, Hkv, page_size)
    one = lambda: (torch.zeros(rows + (D // 2,), dtype=torch.uint8, device=device),  # noqa: E731
                   torch.zeros(rows + (D // 32, 2), dtype=torch.float16, device=device))
    return one() + one()


def _cache(cache, like, Hkv: int, D: int):
    """(pointers, num_pages, page_size) of a cache's arrays, checked."""
    if len(cache) != 4:
        raise ValueError("a cache is (k_codes, k_params, v_codes, v_params)")
    codes = cache[0]
    if not isinstance(codes, torch.Tensor) or codes.dim() != 4:
        raise ValueError("k_codes must be [num_pages, Hkv, page_size, D / 2]")
    rows = (codes.shape[0], Hkv, codes.shape[2])
    for n, side in ((0, "k"), (2, "v")):
        _cuda_tensor(cache[n], side + "_codes", like, torch.uint8, rows + (D // 2,))
        _cuda_tensor(cache[n + 1], side + "_params", like, torch.float16, rows + (D // 32, 2))
    return [t.data_ptr() for t in cache], codes.shape[0], codes.shape[2]


def _pages(page_table, like, B: int) -> int:
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    _cuda_tensor(page_table, "page_table", like, torch.int32, (B, page_table.shape[1]))
    return page_table.shape[1]


def _copy_args(k, v, cache, page_table, start, count):
    _rows16(k, "k")
    B, Hkv, S, D = k.shape
    _cuda_tensor(v, "v", k, k.dtype, k.shape)
    pool, num_pages, page_size = _cache(cache, k, Hkv, D)
    max_pages = _pages(page_table, k, B)
    where = (page_table.data_ptr(), _optional(start, "start", k, torch.int32, (B,)),
             _optional(count, "count", k, torch.int32, (B,)))
    return pool, where, (B, Hkv, S, D, num_pages, page_size, max_pages, _DTYPE[k.dtype])


def fa_cache_write(k, v, cache, page_table, start=None, count=None, stream=None) -> None:
    """Quantises k, v [B, Hkv, S, D] into the 4-bit cache: token i < count[b]
    (default S) of sequence b goes to position start[b] + i (default i) of the
    pages that page_table [B, max_pages] lists."""
    pool, where, sizes = _copy_args(k, v, cache, page_table, start, count)
    with _Call(k, stream) as call:
        st = load().fa_cache_write(k.data_ptr(), v.data_ptr(), *pool, *where, *sizes, call.handle)
    _check(st, "fa_cache_write")


def fa_cache_read(cache, page_table, start=None, count=None, out=None, stream=None):
    """The values of positions start[b] ... start[b] + count[b] - 1 into the
    first rows of ``out`` = (k, v), [B, Hkv, S, D] each; rows past count[b]
    are left as they were.  Returns (k, v)."""
    if out is None or len(out) != 2:
        raise ValueError("out must be the pair (k, v) to read into")
    k, v = out
    pool, where, sizes = _copy_args(k, v, cache, page_table, start, count)
    with _Call(k, stream) as call:
        st = load().fa_cache_read(*pool, *where, k.data_ptr(), v.data_ptr(), *sizes, call.handle)
    _check(st, "fa_cache_read")
    return k, v


def fa_cache_workspace_bytes(B: int, H: int, Hkv: int, Sq: int, D: int, page_size: int,
                             max_pages: int, max_length: int = 0) -> int:
    return int(load().fa_cache_workspace_bytes(B, H, Hkv, Sq, D, page_size, max_pages, max_length))


def fa_fwd_cache(q, cache, page_table, length, scale: float | None = None,
                 softcap: float = 0.0, slopes=None, max_length: int = 0, workspace=None,
                 out=None, lse=None, stream=None):
    """Attention of the newest Sq tokens, q [B, H, Sq, D], over the 4-bit
    cache: length[b] (int32) tokens of sequence b are in it, these included.
    ``max_length``: no sequence is longer (default: what the page table can
    hold); the keys are split over the GPU for it.  Returns (o, lse)."""
    Hkv = cache[0].shape[1] if len(cache) == 4 and cache[0].dim() == 4 else 0
    _grouped(q, Hkv)
    B, H, Sq, D = q.shape
    pool, num_pages, page_size = _cache(cache, q, Hkv, D)
    max_pages = _pages(page_table, q, B)
    _cuda_tensor(length, "length", q, torch.int32, (B,))
    slopes_p = _optional(slopes, "slopes", q, torch.float32, (H,))
    sc = float(D) ** -0.5 if scale is None else float(scale)
    with _Call(q, stream) as call:
        out, lse = _given_outputs(call, q, out, lse)
        need = 0
        if workspace is None:
            need = fa_cache_workspace_bytes(B, H, Hkv, Sq, D, page_size, max_pages, max_length)
        _keep, ws_ptr, ws_bytes = call.workspace(workspace, need)
        st = load().fa_fwd_cache(q.data_ptr(), *pool, page_table.data_ptr(), length.data_ptr(),
                                 out.data_ptr(), lse.data_ptr(), B, H, Hkv, Sq, D, num_pages,
                                 page_size, max_pages, int(max_length), sc, _DTYPE[q.dtype],
                                 float(softcap), slopes_p, ws_ptr, ws_bytes, call.handle)
    _check(st, "fa_fwd_cache")
    return out, lse


def fa_release_workspaces() -> None:
    """Synchronises the device and frees the workspaces fa_fwd keeps for it."""
    _check(load().fa_release_workspaces(), "fa_release_workspaces")


def fa_get_device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word."""
    return int(load().fa_get_device_status(_stream_handle(stream)))


def fa_set_watchdog_ns(ns: int) -> None:
    load().fa_set_watchdog_ns(int(ns))


def fa_status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def fa_prefill_uses_pairs(B: int, H: int, Sq: int, Skv: int, D: int, causal: bool,
                          flags: int = 0, num_splits: int = 0) -> bool:
    return bool(load().fa_prefill_uses_pairs(B, H, Sq, Skv, D, int(bool(causal)), flags,
                                              num_splits))


def fa_prefill_tail_items(B: int, H: int, Sq: int, Skv: int, D: int, causal: bool,
                          dtype=torch.bfloat16, flags: int = 0) -> int:
    """Pair items that fa_fwd_ex with these arguments splits into key
    quarters (FA_FLAG_TAIL_SPLIT); 0 if none."""
    return int(load().fa_prefill_tail_items(B, H, Sq, Skv, D, int(bool(causal)),
                                             _DTYPE[dtype], flags))


def fa_ex2_approx(x, stream=None):
    """2^x on the device with the kernels' exponential instruction (x: a
    contiguous float32 CUDA tensor).  Returns a new tensor."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    y = torch.empty_like(x)
    _check(load().fa_ex2_approx(x.data_ptr(), y.data_ptr(), x.numel(),
                                _stream_handle(stream)), "fa_ex2_approx")
    return y


def fa_version() -> int:
    return int(load().fa_version())
