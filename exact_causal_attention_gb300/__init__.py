"""Exact causal / non-causal attention forward on sm_103a (GB300).

Thin ctypes binding over the C ABI in ``include/attn.h`` and, for the paged cache's
operators, ``include/attn_cache.h``: it checks and marshals
torch tensors into pointers and sizes and calls the library; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if the
shared library is missing or the device is not sm_103, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

__all__ = ["attn_fwd", "attn_fwd_into", "attn_fwd_gqa", "attn_fwd_splitkv", "splitkv_workspace_bytes",
           "splitkv_default_splits", "row_softmax", "decode_paged", "paged_append", "prefill_paged",
           "prefill_workspace_bytes", "paged_append_chunk", "paged_attn_mass", "paged_evict", "load_library", "device_status", "watchdog_selftest", "AttnError",
           "STATUS"]

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libeca_attn.so")
# The same library with the attention kernel's per-CTA milestone stamps compiled in.
ANATOMY_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libeca_attn_anatomy.so")
_lock = threading.Lock()
_lib = None

STATUS = {
    0: "ATTN_OK",
    -1: "ATTN_ERR_INVALID_ARG",
    -2: "ATTN_ERR_UNALIGNED",
    -3: "ATTN_ERR_UNSUPPORTED_D",
    -4: "ATTN_ERR_ARCH",
    -5: "ATTN_ERR_LAUNCH",
    -6: "ATTN_ERR_TIMEOUT",
    -7: "ATTN_ERR_CUDA",
    -8: "ATTN_ERR_SCRATCH_LIMIT",
    -9: "ATTN_ERR_BAD_INDEX",
}

# Every exported symbol of include/attn.h with its ctypes signature.
_VP, _I, _F, _U, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint, ctypes.c_size_t
SIGNATURES = {
    "attn_fwd": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP]),
    "attn_fwd_bf16": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP]),
    "attn_fwd_gqa": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "attn_fwd_gqa_bf16": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP]),
    "attn_fwd_splitkv": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _I, _VP, _SZ, _VP]),
    "attn_fwd_splitkv_bf16": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _I, _VP, _SZ, _VP]),
    "attn_fwd_splitkv_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _I, _VP]),
    "attn_splitkv_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "attn_splitkv_default_splits": (_I, [_I, _I, _I, _I]),
    "attn_row_softmax_f32": (_I, [_VP, _VP, ctypes.c_longlong, _I, _VP]),
    "attn_decode_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _F, _I, _VP, _SZ, _VP]),
    "attn_decode_paged_bf16": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _F, _I, _VP, _SZ,
                                    _VP]),
    "attn_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "attn_decode_default_splits": (_I, [_I, _I, _I, _I, _I]),
    "attn_paged_append": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP]),
    "attn_device_status": (_I, [_VP]),
    "attn_watchdog_selftest": (_I, [_U, _VP]),
    "attn_anatomy_read": (_I, [ctypes.POINTER(ctypes.c_ulonglong), _SZ, _I]),
    "attn_status_string": (ctypes.c_char_p, [_I]),
    "attn_version": (_I, []),
}


# The same for include/attn_cache.h.
_PAGES = [_I] * 4  # D, page_size, max_pages, num_pages
_FORM = [_F, _F, _I, _VP, _VP]  # scale, softcap, window, alibi_slopes, prefix_lens
_PREFILL = [_VP] * 7 + [_I] * 4 + _PAGES + _FORM + [_VP, _SZ, _VP]
_MASS = [_VP] * 7 + [_I] * 5 + _PAGES + _FORM + [_VP]
_DECODE_FORM = [_VP] * 6 + [_I] * 3 + _PAGES + _FORM + [_I, _VP, _SZ, _VP]
CACHE_SIGNATURES = {
    "attn_prefill_paged": (_I, _PREFILL),
    "attn_prefill_paged_bf16": (_I, _PREFILL),
    "attn_prefill_workspace_bytes": (_SZ, [_I] * 7),
    "attn_paged_append_chunk": (_I, [_VP] * 5 + [_I] * 3 + _PAGES + [_VP]),
    "attn_paged_mass": (_I, _MASS),
    "attn_paged_mass_bf16": (_I, _MASS),
    "attn_paged_evict": (_I, [_VP] * 7 + [_I] * 2 + _PAGES + [_I, _I, _VP]),
    "attn_decode_paged_form": (_I, _DECODE_FORM),
    "attn_decode_paged_form_bf16": (_I, _DECODE_FORM),
    "attn_decode_form_default_splits": (_I, [_I] * 5),
}


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_status_text(status)})")


def _status_text(status: int) -> str:
    try:
        return load_library().attn_status_string(status).decode()
    except Exception:  # library missing while formatting an error
        return "?"


def library_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None):
    """Load the CUDA library (built by ``exact_causal_attention_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or _LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"CUDA library not built: {p} is missing "
                                   "(run python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(p)
            for name, (res, args) in [*SIGNATURES.items(), *CACHE_SIGNATURES.items()]:
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check_qkv(q, k, v):
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, H, N, D]")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.shape == k.shape == v.shape):
        raise ValueError("q, k, v must have the same shape [B, H, N, D]")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q, k, v must all be float16 or all bfloat16")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")


_raw_stream_fn = None


def _raw_stream(device_index: int, stream) -> int:
    """cudaStream_t of ``stream``, or of torch's current stream on the device, as an int.
    torch's raw-stream query skips building a Stream object, which costs microseconds."""
    global _raw_stream_fn
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _raw_stream_fn is None:
        import torch

        fn = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream_fn = fn if fn is not None else (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream_fn(device_index)


def _fwd_fast(q, k, v, o, lse, causal, scale, stream) -> bool:
    """The common call, checked with few attribute reads: q, k, v, o contiguous CUDA
    tensors of one shape, 16-bit type and device (the current one), lse None or
    contiguous fp32 [B, H, N] there.  Returns False, having launched nothing, for
    anything else, which the checked path then reports."""
    import torch

    try:
        shape = q.shape
        dt = q.dtype
        dev = q.get_device()
        if (len(shape) != 4 or dev < 0 or dt not in (torch.float16, torch.bfloat16)
                or k.shape != shape or v.shape != shape or o.shape != shape
                or k.dtype != dt or v.dtype != dt or o.dtype != dt
                or k.get_device() != dev or v.get_device() != dev or o.get_device() != dev
                or not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and o.is_contiguous())):
            return False
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != shape[:3] or lse.get_device() != dev
                                or not lse.is_contiguous()):
            return False
        if torch._C._cuda_getDevice() != dev:
            return False
    except (AttributeError, TypeError):
        return False
    B, H, N, D = shape
    lib = load_library()
    fn = lib.attn_fwd_bf16 if dt == torch.bfloat16 else lib.attn_fwd
    rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr() if lse is not None else None,
            B, H, N, D, 1 if causal else 0, 1.0 / math.sqrt(D) if scale is None else float(scale),
            _raw_stream(dev, stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd")
    return True


def attn_fwd_into(q, k, v, o, lse, causal: bool = True, scale: float | None = None, stream=None) -> None:
    """Write O into ``o`` ([B,H,N,D], q's dtype) and the natural-log LSE into ``lse``
    ([B,H,N] float32, or None) on ``stream`` (default: torch's current stream)."""
    import torch

    if _fwd_fast(q, k, v, o, lse, causal, scale, stream):
        return
    _check_qkv(q, k, v)
    B, H, N, D = q.shape
    if o.shape != q.shape or o.dtype != q.dtype or not o.is_contiguous() or o.device != q.device:
        raise ValueError("o must be a contiguous tensor shaped and typed like q")
    if lse is not None and (lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous()
                            or lse.device != q.device):
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor on q's device")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = load_library()
    fn = lib.attn_fwd_bf16 if q.dtype == torch.bfloat16 else lib.attn_fwd
    with torch.cuda.device(q.device):
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                lse.data_ptr() if lse is not None else None, B, H, N, D, int(bool(causal)),
                float(scale), _stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd")


def attn_fwd(q, k, v, causal: bool = True, scale: float | None = None, return_lse: bool = True,
             stream=None):
    """O = softmax(scale * q k^T + mask) v (and the row LSE) for [B, H, N, D] CUDA tensors."""
    import torch

    _check_qkv(q, k, v)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if return_lse else None
    attn_fwd_into(q, k, v, o, lse, causal=causal, scale=scale, stream=stream)
    return (o, lse) if return_lse else o


def attn_fwd_gqa(q, k, v, causal: bool = True, scale: float | None = None, o=None, lse=None, stream=None):
    """Grouped-head attention: q [B,H,N,D], k and v [B,Hkv,N,D] with Hkv dividing H; query head h
    reads key/value head h // (H // Hkv).  Returns (o, lse)."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor")
    B, H, N, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or tuple(k.shape[2:]) != (N, D):
        raise ValueError("k, v must be [B, Hkv, N, D] matching q's B, N, D")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q, k, v must all be float16 or all bfloat16")
    Hkv = k.shape[1]
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = load_library()
    fn = lib.attn_fwd_gqa_bf16 if q.dtype == torch.bfloat16 else lib.attn_fwd_gqa
    with torch.cuda.device(q.device):
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, Hkv, N, D,
                int(bool(causal)), float(scale), _stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_gqa")
    return o, lse


def splitkv_workspace_bytes(B: int, H: int, N: int, D: int, kv_splits: int) -> int:
    """Workspace bytes attn_fwd_splitkv needs (0 for invalid sizes)."""
    return int(load_library().attn_splitkv_workspace_bytes(B, H, N, D, kv_splits))


def splitkv_default_splits(B: int, H: int, N: int, D: int) -> int:
    rc = load_library().attn_splitkv_default_splits(B, H, N, D)
    if rc < 0:
        raise AttnError(rc, "attn_splitkv_default_splits")
    return rc


def attn_fwd_splitkv(q, k, v, o=None, lse=None, kv_splits: int | None = None, workspace=None,
                     causal: bool = True, scale: float | None = None, stream=None):
    """attn_fwd with the key tiles split into kv_splits segments merged by a second
    kernel.  The fp32 workspace comes from the caller (a uint8 CUDA tensor) or is
    allocated here with torch.  Returns (o, lse)."""
    import torch

    _check_qkv(q, k, v)
    B, H, N, D = q.shape
    if kv_splits is None:
        with torch.cuda.device(q.device):
            kv_splits = splitkv_default_splits(B, H, N, D)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    need = splitkv_workspace_bytes(B, H, N, D, kv_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1) + 256, dtype=torch.uint8, device=q.device)
        off = (-workspace.data_ptr()) % 256
        workspace = workspace[off:off + max(need, 1)]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = load_library()
    fn = lib.attn_fwd_splitkv_bf16 if q.dtype == torch.bfloat16 else lib.attn_fwd_splitkv
    with torch.cuda.device(q.device):
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                lse.data_ptr() if lse is not None else None, B, H, N, D, int(bool(causal)), float(scale),
                int(kv_splits), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                _stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_splitkv")
    return o, lse


def row_softmax(x, out=None, stream=None):
    """Row softmax of a contiguous 2-D float32 CUDA tensor (online (m, d) kernel)."""
    import torch

    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2 or x.dtype != torch.float32:
        raise TypeError("x must be a 2-D float32 CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if out is None:
        out = torch.empty_like(x)
    M, N = x.shape
    with torch.cuda.device(x.device):
        rc = load_library().attn_row_softmax_f32(x.data_ptr(), out.data_ptr(), M, N, _stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_row_softmax_f32")
    return out


_torch_module = None


def _torch():
    """torch, imported on first use (an import statement costs a fraction of a microsecond per call)."""
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _check_cache(torch, cache, block_table, lengths):
    """Checks a paged cache with its table and lengths; returns (P, T, Hkv, D, B, max_pages, dtype,
    device index)."""
    shape, table, dt, dev = cache.shape, block_table.shape, cache.dtype, cache.get_device()
    if len(shape) != 5 or shape[1] != 2 or not (dt is torch.float16 or dt is torch.bfloat16):
        raise ValueError("cache must be [P, 2, T, Hkv, D] float16 or bfloat16")
    if len(table) != 2 or lengths.shape != table[:1]:
        raise ValueError("block_table must be [B, max_pages] and lengths [B]")
    if block_table.dtype is not torch.int32 or lengths.dtype is not torch.int32:
        raise ValueError("block_table and lengths must be int32")
    if dev < 0 or block_table.get_device() != dev or lengths.get_device() != dev:
        raise ValueError("cache, block_table and lengths must be CUDA tensors on one device")
    if not (cache.is_contiguous() and block_table.is_contiguous() and lengths.is_contiguous()):
        raise ValueError("cache, block_table and lengths must be contiguous")
    P, _, T, Hkv, D = shape
    B, max_pages = table
    return P, T, Hkv, D, B, max_pages, dt, dev


def _check_like(name: str, t, shape, dtype, dev: int) -> None:
    """``t`` is a contiguous tensor of this shape and dtype on CUDA device ``dev``."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")


def _form_ptrs(alibi_slopes, prefix_lens, Hq: int, B: int, dev: int):
    """Pointers of the optional per-head slopes [Hq] and per-request prefixes [B]."""
    slopes = prefix = None
    if alibi_slopes is not None:
        _check_like("alibi_slopes", alibi_slopes, (Hq,), _torch().float32, dev)
        slopes = alibi_slopes.data_ptr()
    if prefix_lens is not None:
        _check_like("prefix_lens", prefix_lens, (B,), _torch().int32, dev)
        prefix = prefix_lens.data_ptr()
    return slopes, prefix


def _workspace(workspace, need: int, dev: int):
    """(pointer, bytes) of the caller's workspace, or of a new 256-byte aligned one, and
    the tensor that holds it."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _torch().empty(need + 256, dtype=_torch().uint8, device=f"cuda:{dev}")
        ptr = workspace.data_ptr()
        return ptr + (-ptr) % 256, need, workspace
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _call(dev: int, fn, *args) -> int:
    """``fn(*args)`` with CUDA device ``dev`` current."""
    torch = _torch()
    if torch._C._cuda_getDevice() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _within(stream, dev: int):
    """``stream`` as torch's current one: what is allocated inside belongs to it, so that work still
    queued on another stream cannot reach the same memory."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def decode_paged(q, cache, block_table, lengths, scale: float | None = None, kv_splits: int | None = None,
                 out=None, lse=None, workspace=None, stream=None, softcap: float = 0.0, alibi_slopes=None,
                 window: int = 0, prefix_lens=None):
    """One decode step over a paged cache: q [B,Hq,D], cache [P,2,T,Hkv,D] (16-bit),
    block_table [B,max_pages] int32, lengths [B] int32 (all CUDA).  Scores may be capped
    (``softcap``: cap * tanh(s / cap)), biased by distance (``alibi_slopes`` [Hq] float32) and
    limited to the last ``window`` tokens, with the first ``prefix_lens`` [B] int32 tokens
    visible whatever the window.  Returns (out, lse)."""
    torch = _torch()
    B, Hq, D = q.shape
    P, two, T, Hkv, D2 = cache.shape
    if two != 2 or D2 != D or q.dtype != cache.dtype or q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("cache must be [P, 2, T, Hkv, D] in q's dtype")
    if block_table.dtype != torch.int32 or lengths.dtype != torch.int32 or block_table.shape[0] != B:
        raise ValueError("block_table [B, max_pages] and lengths [B] must be int32")
    for t in (q, cache, block_table, lengths):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
    dev = q.get_device()
    if stream is not None and (out is None or lse is None or workspace is None):
        with _within(stream, dev):
            return decode_paged(q, cache, block_table, lengths, scale, kv_splits, out, lse, workspace, None, softcap,
                                alibi_slopes, window, prefix_lens)
    max_pages = block_table.shape[1]
    lib = load_library()
    form = softcap != 0.0 or window != 0 or alibi_slopes is not None or prefix_lens is not None
    if kv_splits is None:
        pick = lib.attn_decode_form_default_splits if form else lib.attn_decode_default_splits
        kv_splits = _call(dev, pick, B, Hq, Hkv, T, max_pages)
        if kv_splits < 0:
            raise AttnError(kv_splits, "attn_decode_default_splits")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = int(lib.attn_decode_workspace_bytes(B, Hq, D, kv_splits))
        if need > 0:
            raw = torch.empty(need + 256, dtype=torch.uint8, device=q.device)
            off = (-raw.data_ptr()) % 256
            workspace = raw[off:off + need]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    sizes = (q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), lengths.data_ptr(), out.data_ptr(),
             lse.data_ptr() if lse is not None else None, B, Hq, Hkv, D, T, max_pages, P, float(scale))
    rest = (int(kv_splits), workspace.data_ptr() if workspace is not None else None,
            (workspace.numel() if workspace is not None else 0), _raw_stream(dev, stream))
    if form:
        slopes, prefix = _form_ptrs(alibi_slopes, prefix_lens, Hq, B, dev)
        fn = lib.attn_decode_paged_form_bf16 if q.dtype == torch.bfloat16 else lib.attn_decode_paged_form
        rc = _call(dev, fn, *sizes, float(softcap), int(window), slopes, prefix, *rest)
    else:
        fn = lib.attn_decode_paged_bf16 if q.dtype == torch.bfloat16 else lib.attn_decode_paged
        rc = _call(dev, fn, *sizes, *rest)
    if rc != 0:
        raise AttnError(rc, "attn_decode_paged")
    return out, lse


def prefill_workspace_bytes(total_q: int, B: int, Hq: int, Hkv: int, D: int, page_size: int, max_pages: int) -> int:
    """Workspace bytes prefill_paged needs (0 for invalid sizes)."""
    return int(load_library().attn_prefill_workspace_bytes(total_q, B, Hq, Hkv, D, page_size, max_pages))


def prefill_paged(q, cache, block_table, lengths, q_offsets, scale: float | None = None, softcap: float = 0.0,
                  alibi_slopes=None, window: int = 0, prefix_lens=None, out=None, lse=None, workspace=None,
                  stream=None):
    """Attention of a ragged chunk of new tokens over a paged cache that already holds their
    K and V: q [total,Hq,D] packed, request b's rows q_offsets[b] .. q_offsets[b+1] - 1 (q_offsets
    [B+1] int32) the last of its lengths[b] tokens; causal; score forms as in decode_paged
    (prefix_lens tokens are visible to every row, earlier ones too).  Rows past q_offsets[B] are
    left alone.  Returns (out, lse [total,Hq] float32)."""
    torch = _torch()
    total, Hq, D = q.shape
    P, T, Hkv, D2, B, max_pages, dt, dev = _check_cache(torch, cache, block_table, lengths)
    if D2 != D:
        raise ValueError("q and cache must have the same head size")
    _check_like("q", q, (total, Hq, D), dt, dev)
    _check_like("q_offsets", q_offsets, (B + 1,), torch.int32, dev)
    slopes, prefix = _form_ptrs(alibi_slopes, prefix_lens, Hq, B, dev)
    if stream is not None and (out is None or lse is None or workspace is None):
        with _within(stream, dev):
            return prefill_paged(q, cache, block_table, lengths, q_offsets, scale, softcap, alibi_slopes, window,
                                 prefix_lens, out, lse, workspace)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like("out", out, (total, Hq, D), dt, dev)
    if lse is None:
        lse = torch.empty((total, Hq), dtype=torch.float32, device=q.device)
    else:
        _check_like("lse", lse, (total, Hq), torch.float32, dev)
    lib = load_library()
    need = 0 if workspace is not None else lib.attn_prefill_workspace_bytes(total, B, Hq, Hkv, D, T, max_pages)
    ws, ws_bytes, held = _workspace(workspace, need, dev)
    fn = lib.attn_prefill_paged_bf16 if dt == torch.bfloat16 else lib.attn_prefill_paged
    rc = _call(dev, fn, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), lengths.data_ptr(),
               q_offsets.data_ptr(), out.data_ptr(), lse.data_ptr(), total, B, Hq, Hkv, D, T, max_pages, P,
               1.0 / math.sqrt(D) if scale is None else float(scale), float(softcap), int(window), slopes, prefix,
               ws, ws_bytes, _raw_stream(dev, stream))
    if rc != 0:
        raise AttnError(rc, "attn_prefill_paged")
    return out, lse


def paged_append_chunk(new_kv, cache, block_table, lengths, q_offsets, stream=None) -> None:
    """Write new_kv [total, 2, Hkv, D], a ragged chunk packed as for prefill_paged, to the last
    positions of every request: its i-th row to lengths[b] - n_b + i."""
    torch = _torch()
    P, T, Hkv, D, B, max_pages, dt, dev = _check_cache(torch, cache, block_table, lengths)
    total = new_kv.shape[0]
    _check_like("new_kv", new_kv, (total, 2, Hkv, D), dt, dev)
    _check_like("q_offsets", q_offsets, (B + 1,), torch.int32, dev)
    rc = _call(dev, load_library().attn_paged_append_chunk, new_kv.data_ptr(), cache.data_ptr(),
               block_table.data_ptr(), lengths.data_ptr(), q_offsets.data_ptr(), total, B, Hkv, D, T, max_pages, P,
               _raw_stream(dev, stream))
    if rc != 0:
        raise AttnError(rc, "attn_paged_append_chunk")


def paged_attn_mass(q, lse, cache, block_table, lengths, q_offsets=None, mass=None, scale: float | None = None,
                    softcap: float = 0.0, alibi_slopes=None, window: int = 0, prefix_lens=None, stream=None):
    """The attention weight every cached token received from the rows of q [total,Hq,D] (packed as
    for prefill_paged, or one row a request when q_offsets is None), whose log-sum-exps lse
    [total,Hq] came from prefill_paged or decode_paged with the same score form: summed over the
    rows and the query heads of each key/value head.  Added to ``mass`` [B,Hkv,max_pages*T] float32
    when given, else written to a new one.  Returns mass."""
    torch = _torch()
    total, Hq, D = q.shape
    P, T, Hkv, D2, B, max_pages, dt, dev = _check_cache(torch, cache, block_table, lengths)
    if D2 != D:
        raise ValueError("q and cache must have the same head size")
    _check_like("q", q, (total, Hq, D), dt, dev)
    _check_like("lse", lse, (total, Hq), torch.float32, dev)
    offsets = None
    if q_offsets is not None:
        _check_like("q_offsets", q_offsets, (B + 1,), torch.int32, dev)
        offsets = q_offsets.data_ptr()
    elif total != B:
        raise ValueError("without q_offsets q holds one row a request")
    slopes, prefix = _form_ptrs(alibi_slopes, prefix_lens, Hq, B, dev)
    accumulate = mass is not None
    if stream is not None and not accumulate:
        with _within(stream, dev):
            return paged_attn_mass(q, lse, cache, block_table, lengths, q_offsets, None, scale, softcap, alibi_slopes,
                                   window, prefix_lens)
    if accumulate:
        _check_like("mass", mass, (B, Hkv, max_pages * T), torch.float32, dev)
    else:
        mass = torch.empty((B, Hkv, max_pages * T), dtype=torch.float32, device=q.device)
    lib = load_library()
    fn = lib.attn_paged_mass_bf16 if dt == torch.bfloat16 else lib.attn_paged_mass
    rc = _call(dev, fn, q.data_ptr(), lse.data_ptr(), cache.data_ptr(), block_table.data_ptr(), lengths.data_ptr(),
               offsets, mass.data_ptr(), int(accumulate), total, B, Hq, Hkv, D, T, max_pages, P,
               1.0 / math.sqrt(D) if scale is None else float(scale), float(softcap), int(window), slopes, prefix,
               _raw_stream(dev, stream))
    if rc != 0:
        raise AttnError(rc, "attn_paged_mass")
    return mass


def paged_evict(cache, block_table, lengths, mass, budget: int, recent: int = 0, kept=None, new_lengths=None,
                mass_out=None, stream=None):
    """Shrink every request that holds more than ``budget`` tokens to ``budget`` of them, per
    key/value head: the last ``recent`` tokens and, of the others, those with the largest mass
    [B,Hkv,max_pages*T] float32 (ties: the lowest position).  Their rows move in place to positions
    0 .. budget - 1, in order.  Returns (kept [B,Hkv,budget] int32: each one's old position, then
    -1; new_lengths [B] int32; mass_out: the kept tokens' mass, then 0)."""
    torch = _torch()
    P, T, Hkv, D, B, max_pages, _, dev = _check_cache(torch, cache, block_table, lengths)
    _check_like("mass", mass, (B, Hkv, max_pages * T), torch.float32, dev)
    budget = int(budget)
    if stream is not None and (kept is None or new_lengths is None or mass_out is None):
        with _within(stream, dev):
            return paged_evict(cache, block_table, lengths, mass, budget, recent, kept, new_lengths, mass_out)
    if kept is None:
        kept = torch.empty((B, Hkv, max(budget, 0)), dtype=torch.int32, device=cache.device)
    else:
        _check_like("kept", kept, (B, Hkv, budget), torch.int32, dev)
    if new_lengths is None:
        new_lengths = torch.empty_like(lengths)
    else:
        _check_like("new_lengths", new_lengths, (B,), torch.int32, dev)
    if mass_out is None:
        mass_out = torch.empty_like(mass)
    else:
        _check_like("mass_out", mass_out, (B, Hkv, max_pages * T), torch.float32, dev)
    rc = _call(dev, load_library().attn_paged_evict, cache.data_ptr(), block_table.data_ptr(), lengths.data_ptr(),
               mass.data_ptr(), kept.data_ptr(), new_lengths.data_ptr(), mass_out.data_ptr(), B, Hkv, D, T, max_pages,
               P, budget, int(recent), _raw_stream(dev, stream))
    if rc != 0:
        raise AttnError(rc, "attn_paged_evict")
    return kept, new_lengths, mass_out


def paged_append(new_kv, cache, block_table, lengths, stream=None) -> None:
    """Write new_kv [B, 2, Hkv, D] at position lengths[b] - 1 of every request's pages."""
    import torch

    B, two, Hkv, D = new_kv.shape
    P, _, T, _, _ = cache.shape
    with torch.cuda.device(cache.device):
        rc = load_library().attn_paged_append(new_kv.data_ptr(), cache.data_ptr(), block_table.data_ptr(),
                                              lengths.data_ptr(), B, Hkv, D, T, block_table.shape[1], P,
                                              _stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_paged_append")


def device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status word (0 = ok)."""
    return load_library().attn_device_status(_stream_handle(stream))


def watchdog_selftest(timeout_us: int, stream=None) -> None:
    rc = load_library().attn_watchdog_selftest(int(timeout_us), _stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_watchdog_selftest")
