"""ctypes binding of ``libfp_serve.so`` (the C ABI in ``include/fp_serve.h``):
sliding-window attention with sink tokens, the paged key/value cache and the
attention of new tokens over it.

Two layers, as in ``ops``, argument marshalling only:

* ``fp_*`` functions with the C names and the C argument order; tensors are
  passed as device pointers, the stream defaults to torch's current stream.
* ``window_attn``, ``kv_write``, ``kv_read`` and ``paged_attn``, which check
  their tensors, create the outputs and the workspace with torch and call the
  ``fp_*`` function on the tensors' device.  A serving loop makes a ``KVCache``
  and a ``Batch`` once: they hold tensors, whose contents (lengths, pages) may
  change between calls, also between replays of a captured call.

The library is loaded on first use; if it is missing this raises instead of
falling back to anything else.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re

import torch

from . import build as _build
from . import ops
from .ops import FP_BF16, FP_F32, FPError, fp_shape  # noqa: F401

FP_E4M3 = 2
HEADER = os.path.join(os.path.dirname(ops.HEADER), "fp_serve.h")
_DTYPES = {torch.bfloat16: FP_BF16, torch.float32: FP_F32, torch.float8_e4m3fn: FP_E4M3}
_P, _I, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


class fp_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", _I), ("n_kv_heads", _I), ("page_size", _I), ("head_dim", _I),
                ("dtype", _I), ("k", _P), ("v", _P), ("k_exps", _P), ("v_exps", _P)]


class fp_batch(ctypes.Structure):
    _fields_ = [("n_seqs", _I), ("max_pages", _I), ("max_q_len", _I), ("total_q", _I),
                ("page_table", _P), ("kv_lens", _P), ("q_offsets", _P)]


_SIG = {
    "fp_window_attn": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "fp_kv_write": (_I, [_P, _P, _I, _P, _P, _P]),
    "fp_kv_read": (_I, [_P, _P, _I, _P, _P, _P]),
    "fp_paged_attn_workspace": (_Z, [_P, _P, _I]),
    "fp_paged_attn": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "fp_serve_last_device_status": (_I, [_P]),
}

_LIB = None


def lib_path() -> str:
    return os.environ.get("FP_SERVE_LIBRARY", _build.SERVE_LIB)


def lib() -> ctypes.CDLL:
    """The loaded library (raises RuntimeError if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "(there is no fallback implementation)")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIG.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def header_functions() -> list[str]:
    """Names of the functions declared in include/fp_serve.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:fp_status|size_t)\s*(fp_\w+)\s*\(", text, re.M)))


# ------------------------------------------------------------------ marshal --

def _ref(x):
    return None if x is None else ctypes.byref(x)


def _stream(stream):
    if stream is None and torch.cuda.is_initialized():
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return ops._stream(stream)


def fp_window_attn(shape, window, sinks, q, k, v, out, lse, stream=None) -> int:
    return lib().fp_window_attn(_ref(shape), window, sinks, ops._addr(q), ops._addr(k),
                                ops._addr(v), ops._addr(out), ops._addr(lse),
                                _stream(stream))


def fp_kv_write(cache, batch, dtype, k, v, stream=None) -> int:
    return lib().fp_kv_write(_ref(cache), _ref(batch), dtype, ops._addr(k), ops._addr(v),
                             _stream(stream))


def fp_kv_read(cache, batch, dtype, k, v, stream=None) -> int:
    return lib().fp_kv_read(_ref(cache), _ref(batch), dtype, ops._addr(k), ops._addr(v),
                            _stream(stream))


def fp_paged_attn_workspace(cache, batch, n_q_heads) -> int:
    return int(lib().fp_paged_attn_workspace(_ref(cache), _ref(batch), n_q_heads))


def fp_paged_attn(cache, batch, n_q_heads, dtype, window, sinks, q, out, lse, ws,
                  stream=None) -> int:
    return lib().fp_paged_attn(_ref(cache), _ref(batch), n_q_heads, dtype, window, sinks,
                               ops._addr(q), ops._addr(out), ops._addr(lse), ops._addr(ws),
                               ops._nbytes(ws), _stream(stream))


def fp_serve_last_device_status(stream=None) -> int:
    return lib().fp_serve_last_device_status(_stream(stream))


# ------------------------------------------------------------- descriptions --

def _need(x, name, dtypes, device=None, dim=None) -> None:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {x.dtype}")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    if dim is not None and x.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class KVCache:
    """A paged cache over the caller's tensors: k, v [n_pages, Hkv, page_size, d]
    (bf16, fp32 or float8_e4m3fn) and, for 8 bits, the exponent bytes k_exps,
    v_exps [n_pages, Hkv, page_size] (uint8).  ``kv_cache`` allocates one."""

    def __init__(self, k, v, k_exps=None, v_exps=None):
        _need(k, "k", _DTYPES, dim=4)
        _need(v, "v", (k.dtype,), k.device, dim=4)
        if v.shape != k.shape:
            raise ValueError("k and v must have one shape")
        narrow = k.dtype == torch.float8_e4m3fn
        if (k_exps is not None or v_exps is not None) != narrow or (k_exps is None) != (
                v_exps is None):
            raise ValueError("k_exps and v_exps belong to an 8-bit cache, both of them")
        for name, x in (("k_exps", k_exps), ("v_exps", v_exps)):
            if x is not None:
                _need(x, name, (torch.uint8,), k.device, dim=3)
                if x.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be {tuple(k.shape[:3])}")
        self.k, self.v, self.k_exps, self.v_exps = k, v, k_exps, v_exps
        self.device, self.dtype = k.device, k.dtype
        pages, heads, size, d = k.shape
        self.struct = fp_kv_cache(pages, heads, size, d, _DTYPES[k.dtype], k.data_ptr(),
                                  v.data_ptr(), _ptr(k_exps), _ptr(v_exps))
        self.ref = ctypes.byref(self.struct)


def kv_cache(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int,
             dtype=torch.bfloat16, device="cuda") -> KVCache:
    """A new, uninitialised cache."""
    shape = (n_pages, n_kv_heads, page_size, head_dim)
    k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.empty(shape[:3], dtype=torch.uint8, device=device)
                           for _ in range(2)))


class Batch:
    """Sequences and their newest tokens (``fp_batch``): page_table int32
    [n_seqs, max_pages], kv_lens int32 [n_seqs] (the new tokens included) and
    q_offsets int32 [n_seqs + 1], or None where every sequence has max_q_len new
    tokens.  With q_offsets, total_q is the number of rows per head that the
    packed tensors hold (q_offsets[-1] or more)."""

    def __init__(self, page_table, kv_lens, q_offsets=None, max_q_len: int = 1,
                 total_q: int | None = None):
        _need(page_table, "page_table", (torch.int32,), dim=2)
        device = page_table.device
        n = page_table.shape[0]
        for name, x, want in (("kv_lens", kv_lens, n), ("q_offsets", q_offsets, n + 1)):
            if x is None and name == "q_offsets":
                continue
            _need(x, name, (torch.int32,), device, dim=1)
            if x.shape[0] != want:
                raise ValueError(f"{name} must have {want} entries")
        if q_offsets is None:
            if total_q is not None and total_q != n * max_q_len:
                raise ValueError("without q_offsets, total_q is n_seqs * max_q_len")
            total_q = n * max_q_len
        elif total_q is None:
            raise ValueError("q_offsets needs total_q")
        self.page_table, self.kv_lens, self.q_offsets = page_table, kv_lens, q_offsets
        self.device, self.max_q_len, self.total_q = device, max_q_len, total_q
        self.struct = fp_batch(n, page_table.shape[1], max_q_len, total_q,
                               page_table.data_ptr(), kv_lens.data_ptr(), _ptr(q_offsets))
        self.ref = ctypes.byref(self.struct)


# ------------------------------------------------------------------ helpers --

@contextlib.contextmanager
def _elsewhere(device, stream):
    """Makes `device` and `stream` the current ones, so that outputs and
    workspaces are allocated where they are used."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            yield


def _here(device, stream) -> bool:
    return stream is None and device.index == torch.cuda.current_device()


def _raw_stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(x):
    return None if x is None else x.data_ptr()


def _packed(x, name, cache, batch, heads, dtypes) -> int:
    """Checks a packed tensor [.., d] and returns its number of heads."""
    _need(x, name, dtypes, cache.device)
    if batch.device != cache.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    d = cache.struct.head_dim
    if x.dim() < 2 or x.shape[-1] != d:
        raise ValueError(f"{name} must end in the cache's head dimension {d}")
    rows = x.numel() // d
    if heads is None:
        heads = rows // batch.total_q if batch.total_q else cache.struct.n_kv_heads
    if rows != heads * batch.total_q:
        raise ValueError(f"{name} must hold total_q rows per head")
    return heads


def workspace(cache: KVCache, batch: Batch, n_q_heads: int) -> torch.Tensor | None:
    """A device byte buffer of fp_paged_attn_workspace bytes, or None if 0 (fp32
    queries need none)."""
    n = lib().fp_paged_attn_workspace(cache.ref, batch.ref, n_q_heads)
    return torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None


def _buffer(ws, device) -> None:
    """Refuses a workspace that is not a plain buffer on `device` (an expanded view
    says more bytes than it has)."""
    if not isinstance(ws, torch.Tensor) or ws.device != device:
        raise ValueError(f"the workspace must be a tensor on {device}")
    if not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous")


# -------------------------------------------------------------------- calls --

def window_attn(q, k, v, window: int, sinks: int = 0, with_lse: bool = True, stream=None):
    """fp_window_attn: causal attention in which a query sees the last `window`
    keys (<= 0: all) and the first `sinks`; q [Bt, Hq, N, d], k and v
    [Bt, Hkv, N, d].  (out like q, lse fp32 [Bt, Hq, N] or None)."""
    _need(q, "q", (torch.bfloat16, torch.float32), dim=4)
    device = q.device
    bt, hq, n, d = q.shape
    for name, x in (("k", k), ("v", v)):
        _need(x, name, (q.dtype,), device, dim=4)
        if x.shape[0] != bt or x.shape[2] != n or x.shape[3] != d or x.shape[1] != k.shape[1]:
            raise ValueError(f"{name} does not fit q")
    if not _here(device, stream):
        with _elsewhere(device, stream):
            return window_attn(q, k, v, window, sinks, with_lse)
    s = fp_shape(bt, hq, k.shape[1], n, d, 128, _DTYPES[q.dtype])
    out = torch.empty_like(q)
    lse = q.new_empty((bt, hq, n), dtype=torch.float32) if with_lse else None
    ops._check(lib().fp_window_attn(ctypes.byref(s), window, sinks, q.data_ptr(), k.data_ptr(),
                                    v.data_ptr(), out.data_ptr(), _ptr(lse),
                                    _raw_stream(device)), "fp_window_attn")
    return out, lse


def kv_write(cache: KVCache, batch: Batch, k, v, stream=None) -> None:
    """fp_kv_write: stores the new tokens' packed k and v ([Bt, Hkv, N, d], or
    the sequences' [Hkv, n_s, d] back to back as rows of d)."""
    dtypes = (torch.bfloat16, torch.float32)
    if cache.dtype in dtypes:
        dtypes = (cache.dtype,)
    _packed(k, "k", cache, batch, cache.struct.n_kv_heads, dtypes)
    _packed(v, "v", cache, batch, cache.struct.n_kv_heads, (k.dtype,))
    if not _here(cache.device, stream):
        with _elsewhere(cache.device, stream):
            return kv_write(cache, batch, k, v)
    ops._check(lib().fp_kv_write(cache.ref, batch.ref, _DTYPES[k.dtype], k.data_ptr(),
                                 v.data_ptr(), _raw_stream(cache.device)), "fp_kv_write")


def kv_read(cache: KVCache, batch: Batch, dtype=None, stream=None):
    """fp_kv_read: (k, v) of the newest tokens, [n_seqs, Hkv, max_q_len, d] or,
    with q_offsets, packed rows [total_q * Hkv, d]; dtype defaults to the
    cache's (bf16 from 8 bits)."""
    if dtype is None:
        dtype = torch.bfloat16 if cache.dtype == torch.float8_e4m3fn else cache.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}")
    if batch.device != cache.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    if not _here(cache.device, stream):
        with _elsewhere(cache.device, stream):
            return kv_read(cache, batch, dtype)
    heads, d = cache.struct.n_kv_heads, cache.struct.head_dim
    shape = (batch.total_q * heads, d)
    if batch.q_offsets is None:
        shape = (batch.struct.n_seqs, heads, batch.max_q_len, d)
    k = cache.k.new_empty(shape, dtype=dtype)
    v = torch.empty_like(k)
    ops._check(lib().fp_kv_read(cache.ref, batch.ref, _DTYPES[dtype], k.data_ptr(),
                                v.data_ptr(), _raw_stream(cache.device)), "fp_kv_read")
    return k, v


def paged_attn(q, cache: KVCache, batch: Batch, window: int = 0, sinks: int = 0,
               with_lse: bool = True, ws=None, stream=None):
    """fp_paged_attn: the new tokens' packed queries ([Bt, Hq, N, d], or the
    sequences' [Hq, n_s, d] back to back as rows of d) attend to their
    sequences in the cache.  (out like q, lse fp32 [..] or None)."""
    heads = _packed(q, "q", cache, batch, None, (torch.bfloat16, torch.float32))
    device = cache.device
    if not _here(device, stream):
        with _elsewhere(device, stream):
            return paged_attn(q, cache, batch, window, sinks, with_lse, ws)
    out = torch.empty_like(q)
    lse = q.new_empty(q.shape[:-1], dtype=torch.float32) if with_lse else None
    if ws is not None:
        _buffer(ws, device)
    elif q.dtype != torch.float32:
        ws = workspace(cache, batch, heads)
    ops._check(lib().fp_paged_attn(cache.ref, batch.ref, heads, _DTYPES[q.dtype], window, sinks,
                                   q.data_ptr(), out.data_ptr(), _ptr(lse), _ptr(ws),
                                   ops._nbytes(ws), _raw_stream(device)), "fp_paged_attn")
    return out, lse
