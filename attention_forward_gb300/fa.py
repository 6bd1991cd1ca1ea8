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
    L.fa_score_item_rows.argtypes = [ci] * 6
    L.fa_score_item_rows.restype = ci
    L.fa_score_key_ranges.argtypes = [ci] * 6
    L.fa_score_key_ranges.restype = ci
    L.fa_fwd_score.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, cf,
                               vp, vp, vp, vp, vp, sz, vp]
    L.fa_fwd_score.restype = ci
    L.fa_cache_write.argtypes = [vp] * 9 + [ci] * 8 + [vp]
    L.fa_cache_write.restype = ci
    L.fa_cache_read.argtypes = [vp] * 9 + [ci] * 8 + [vp]
    L.fa_cache_read.restype = ci
    L.fa_cache_workspace_bytes.argtypes = [ci] * 7
    L.fa_cache_workspace_bytes.restype = sz
    L.fa_fwd_cache.argtypes = [vp] * 9 + [ci] * 8 + [cf, ci, cf, vp, vp, sz, vp]
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


# The raw handle of a device's current stream, without making a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _own_memory(tensors, stream) -> None:
    """Memory made on the current stream for work on another one: that stream
    waits for the work that last had it, and the memory outlives the call's."""
    handle = _stream_handle(stream)
    if handle != _raw_stream(_current_device()):
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(handle)
        stream.wait_stream(torch.cuda.current_stream())
        for t in tensors:
            t.record_stream(stream)


def _bad(t, name: str, dev: int, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a tensor on the call's CUDA device")
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _ptr(t, name: str, dev: int, dtype, shape) -> int:
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass  # not a tensor
    _bad(t, name, dev, dtype, shape)


def _rows16(t, name: str):
    """(device, shape) of a 4-d 16-bit CUDA tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be a 4-d float16 or bfloat16 tensor")
    dev = t.get_device()
    if dev < 0 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return dev, t.shape


def _group_check(H: int, Hkv: int) -> None:
    if Hkv < 1 or H % Hkv != 0:
        raise ValueError("the kv heads must divide the query heads")


def _outputs_on(q, dev, out, lse, stream):
    """The outputs of a call on q's device, made where they are not given."""
    B, H, Sq, D = q.shape
    if out is None and lse is None and stream is None:
        return (torch.empty_like(q),
                torch.empty((B, H, Sq), dtype=torch.float32, device=q.device))
    made = []
    if out is None:
        out = torch.empty_like(q)
        made.append(out)
    else:
        _ptr(out, "out", dev, q.dtype, q.shape)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
        made.append(lse)
    else:
        _ptr(lse, "lse", dev, torch.float32, (B, H, Sq))
    if stream is not None and made:
        _own_memory(made, stream)
    return out, lse


def _workspace_of(workspace, dev):
    """(pointer, bytes) of a caller's workspace."""
    if workspace.get_device() != dev or not workspace.is_contiguous() or not workspace.numel():
        raise ValueError("workspace must be a contiguous tensor on the call's CUDA device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _graph_workspace(call, need: int, device, stream) -> int:
    """Repeats a captured call, which may not use the library's workspace, with
    one of the graph's own memory."""
    workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if stream is not None:
        _own_memory([workspace], stream)
    return call(workspace.data_ptr(), need)


def fa_score_workspace_bytes(B: int, H: int, Hkv: int, Sq: int, Skv: int, D: int,
                             documents: bool = False) -> int:
    return int(load().fa_score_workspace_bytes(B, H, Hkv, Sq, Skv, D, int(bool(documents))))


def fa_score_item_rows(B: int, H: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    """Rows of a work item of fa_fwd_score at these sizes: 256, or 128 whose key
    tiles an item's two stages share."""
    return int(load().fa_score_item_rows(B, H, Hkv, Sq, Skv, D))


def fa_score_key_ranges(B: int, H: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    """Ranges that fa_fwd_score splits an item's keys into at these sizes."""
    return int(load().fa_score_key_ranges(B, H, Hkv, Sq, Skv, D))


def fa_fwd_score(q, k, v, causal: bool = False, scale: float | None = None,
                 softcap: float = 0.0, slopes=None, doc_q=None, doc_k=None, prefix=None,
                 workspace=None, out=None, lse=None, stream=None):
    """Attention with modified scores on grouped heads: q [B, H, Sq, D], k and
    v [B, Hkv, Skv, D].  ``softcap`` caps the scores by a tanh, ``slopes``
    (float32 [H]) takes slope * distance off them, ``doc_q`` / ``doc_k``
    (int32 [B, Sq], [B, Skv]) keep rows to keys of their document, ``prefix``
    (int32 [B], causal only) shows the first keys to every row.  In bfloat16
    under a cap of at most 50, v is taken up to 2^30 in magnitude (below 2^-50 it
    may count as 0), unless ``slopes``, zeros if need be, are given.  Without
    ``workspace`` the library's own for the stream serves (a captured call gets
    one of the graph's memory).  Returns (o, lse)."""
    dev, (B, H, Sq, D) = _rows16(q, "q")
    _, kv = _rows16(k, "k")
    Hkv, Skv = kv[1], kv[2]
    _group_check(H, Hkv)
    if kv[0] != B or kv[3] != D or k.dtype is not q.dtype or k.get_device() != dev:
        _bad(k, "k", dev, q.dtype, (B, Hkv, Skv, D))
    kp, vp = k.data_ptr(), _ptr(v, "v", dev, q.dtype, kv)
    sp = dqp = dkp = pp = None
    if slopes is not None:
        sp = _ptr(slopes, "slopes", dev, torch.float32, (H,))
    if doc_q is not None:
        dqp = _ptr(doc_q, "doc_q", dev, torch.int32, (B, Sq))
    if doc_k is not None:
        dkp = _ptr(doc_k, "doc_k", dev, torch.int32, (B, Skv))
    if prefix is not None:
        pp = _ptr(prefix, "prefix", dev, torch.int32, (B,))
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return fa_fwd_score(q, k, v, causal, scale, softcap, slopes, doc_q, doc_k, prefix,
                                workspace, out, lse, stream)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    L = _lib or load()
    out, lse = _outputs_on(q, dev, out, lse, stream)
    ws, ws_bytes = (None, 0) if workspace is None else _workspace_of(workspace, dev)
    args = (q.data_ptr(), kp, vp, out.data_ptr(), lse.data_ptr(), B, H, Hkv, Sq, Skv, D, sc,
            bool(causal), _DTYPE[q.dtype], softcap, sp, dqp, dkp, pp)
    handle = _raw_stream(dev) if stream is None else _stream_handle(stream)
    if ws is None and torch.cuda.is_current_stream_capturing():
        need = L.fa_score_workspace_bytes(B, H, Hkv, Sq, Skv, D, doc_k is not None)
        st = _graph_workspace(lambda p, n: L.fa_fwd_score(*args, p, n, handle), need, q.device,
                              stream)
    else:
        st = L.fa_fwd_score(*args, ws, ws_bytes, handle)
    if st:
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


def _cache(cache, dev: int, Hkv: int, D: int):
    """A cache's four pointers, num_pages and page_size, checked."""
    if len(cache) != 4:
        raise ValueError("a cache is (k_codes, k_params, v_codes, v_params)")
    kc, kp, vc, vp = cache
    if not isinstance(kc, torch.Tensor) or kc.dim() != 4:
        raise ValueError("k_codes must be [num_pages, Hkv, page_size, D / 2]")
    pages, _, page, _ = kc.shape
    codes, params = (pages, Hkv, page, D // 2), (pages, Hkv, page, D // 32, 2)
    return (_ptr(kc, "k_codes", dev, torch.uint8, codes),
            _ptr(kp, "k_params", dev, torch.float16, params),
            _ptr(vc, "v_codes", dev, torch.uint8, codes),
            _ptr(vp, "v_params", dev, torch.float16, params), pages, page)


def _pages(page_table, dev: int, B: int):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    n = page_table.shape[1]
    return _ptr(page_table, "page_table", dev, torch.int32, (B, n)), n


def _copy_args(k, v, cache, page_table, start, count):
    """(device, arguments) of a cache copy.  The checks in one expression, for
    their time beside the copies' own; what it refuses is named one by one."""
    try:
        kc, kp, vc, vp = cache
        dt, rows, dev = k.dtype, k.shape, k.get_device()
        B, Hkv, S, D = rows
        pages, _, page, _ = kc.shape
        n, per = page_table.shape
        codes, params = (pages, Hkv, page, D // 2), (pages, Hkv, page, D // 32, 2)
        u8, f16, i32 = torch.uint8, torch.float16, torch.int32
        if (dev >= 0 and k.is_contiguous() and n == B
                and v.dtype is dt and v.shape == rows and v.get_device() == dev
                and v.is_contiguous()
                and kc.dtype is u8 and kc.shape == codes and kc.get_device() == dev
                and kc.is_contiguous()
                and kp.dtype is f16 and kp.shape == params and kp.get_device() == dev
                and kp.is_contiguous()
                and vc.dtype is u8 and vc.shape == codes and vc.get_device() == dev
                and vc.is_contiguous()
                and vp.dtype is f16 and vp.shape == params and vp.get_device() == dev
                and vp.is_contiguous()
                and page_table.dtype is i32 and page_table.get_device() == dev
                and page_table.is_contiguous()
                and (start is None or start.dtype is i32 and start.shape == (B,)
                     and start.get_device() == dev and start.is_contiguous())
                and (count is None or count.dtype is i32 and count.shape == (B,)
                     and count.get_device() == dev and count.is_contiguous())):
            return (dev, (k.data_ptr(), v.data_ptr()),
                    (kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr()),
                    (page_table.data_ptr(), None if start is None else start.data_ptr(),
                     None if count is None else count.data_ptr()),
                    (B, Hkv, S, D, pages, page, per, _DTYPE[dt]))
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        pass
    dev, (B, Hkv, S, D) = _rows16(k, "k")
    vptr = _ptr(v, "v", dev, k.dtype, k.shape)
    kc, kp, vc, vp, pages, page = _cache(cache, dev, Hkv, D)
    table, per = _pages(page_table, dev, B)
    if start is not None:
        start = _ptr(start, "start", dev, torch.int32, (B,))
    if count is not None:
        count = _ptr(count, "count", dev, torch.int32, (B,))
    return (dev, (k.data_ptr(), vptr), (kc, kp, vc, vp), (table, start, count),
            (B, Hkv, S, D, pages, page, per, _DTYPE[k.dtype]))


def fa_cache_write(k, v, cache, page_table, start=None, count=None, stream=None) -> None:
    """Quantises k, v [B, Hkv, S, D] into the 4-bit cache: token i < count[b]
    (default S) of sequence b goes to position start[b] + i (default i) of the
    pages that page_table [B, max_pages] lists."""
    dev, rows, pool, where, sizes = _copy_args(k, v, cache, page_table, start, count)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return fa_cache_write(k, v, cache, page_table, start, count, stream)
    st = (_lib or load()).fa_cache_write(
        *rows, *pool, *where, *sizes,
        _raw_stream(dev) if stream is None else _stream_handle(stream))
    if st:
        _check(st, "fa_cache_write")


def fa_cache_read(cache, page_table, start=None, count=None, out=None, stream=None):
    """The values of positions start[b] ... start[b] + count[b] - 1 into the
    first rows of ``out`` = (k, v), [B, Hkv, S, D] each; rows past count[b]
    are left as they were.  Returns (k, v)."""
    if out is None or len(out) != 2:
        raise ValueError("out must be the pair (k, v) to read into")
    k, v = out
    dev, rows, pool, where, sizes = _copy_args(k, v, cache, page_table, start, count)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return fa_cache_read(cache, page_table, start, count, out, stream)
    st = (_lib or load()).fa_cache_read(
        *pool, *where, *rows, *sizes,
        _raw_stream(dev) if stream is None else _stream_handle(stream))
    if st:
        _check(st, "fa_cache_read")
    return k, v


def fa_cache_workspace_bytes(B: int, H: int, Hkv: int, Sq: int, D: int, page_size: int,
                             max_pages: int) -> int:
    return int(load().fa_cache_workspace_bytes(B, H, Hkv, Sq, D, page_size, max_pages))


def _attn_args(cache, page_table, length, dev: int, B: int, H: int, D: int):
    """As _copy_args: a cache, its page table and lengths."""
    try:
        kc, kp, vc, vp = cache
        pages, Hkv, page, _ = kc.shape
        n, per = page_table.shape
        codes, params = (pages, Hkv, page, D // 2), (pages, Hkv, page, D // 32, 2)
        u8, f16, i32 = torch.uint8, torch.float16, torch.int32
        if (n == B and Hkv > 0 and H % Hkv == 0
                and kc.dtype is u8 and kc.shape == codes and kc.get_device() == dev
                and kc.is_contiguous()
                and kp.dtype is f16 and kp.shape == params and kp.get_device() == dev
                and kp.is_contiguous()
                and vc.dtype is u8 and vc.shape == codes and vc.get_device() == dev
                and vc.is_contiguous()
                and vp.dtype is f16 and vp.shape == params and vp.get_device() == dev
                and vp.is_contiguous()
                and page_table.dtype is i32 and page_table.get_device() == dev
                and page_table.is_contiguous()
                and length.dtype is i32 and length.shape == (B,)
                and length.get_device() == dev and length.is_contiguous()):
            return (Hkv, kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), pages, page,
                    page_table.data_ptr(), per, length.data_ptr())
    except (AttributeError, IndexError, TypeError, ValueError):
        pass
    Hkv = cache[0].shape[1] if len(cache) == 4 and cache[0].dim() == 4 else 0
    _group_check(H, Hkv)
    kc, kp, vc, vp, pages, page = _cache(cache, dev, Hkv, D)
    table, per = _pages(page_table, dev, B)
    return (Hkv, kc, kp, vc, vp, pages, page, table, per,
            _ptr(length, "length", dev, torch.int32, (B,)))


def fa_fwd_cache(q, cache, page_table, length, scale: float | None = None,
                 softcap: float = 0.0, slopes=None, workspace=None, out=None, lse=None,
                 stream=None):
    """Attention of the newest Sq tokens, q [B, H, Sq, D], over the 4-bit
    cache: length[b] (int32) tokens of sequence b are in it, these included.
    Returns (o, lse)."""
    dev, (B, H, Sq, D) = _rows16(q, "q")
    ptrs = _attn_args(cache, page_table, length, dev, B, H, D)
    Hkv, kc, kp, vc, vp, pages, page, table, per, lp = ptrs
    sp = None
    if slopes is not None:
        sp = _ptr(slopes, "slopes", dev, torch.float32, (H,))
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return fa_fwd_cache(q, cache, page_table, length, scale, softcap, slopes, workspace,
                                out, lse, stream)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    L = _lib or load()
    out, lse = _outputs_on(q, dev, out, lse, stream)
    ws, ws_bytes = (None, 0) if workspace is None else _workspace_of(workspace, dev)
    args = (q.data_ptr(), kc, kp, vc, vp, table, lp, out.data_ptr(), lse.data_ptr(), B, H, Hkv,
            Sq, D, pages, page, per, sc, _DTYPE[q.dtype], softcap, sp)
    handle = _raw_stream(dev) if stream is None else _stream_handle(stream)
    st = L.fa_fwd_cache(*args, ws, ws_bytes, handle)
    if st == FA_ERR_WORKSPACE and ws is None:
        need = L.fa_cache_workspace_bytes(B, H, Hkv, Sq, D, page, per)
        st = _graph_workspace(lambda p, n: L.fa_fwd_cache(*args, p, n, handle), need, q.device,
                              stream)
    if st:
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
