"""The paged key/value cache in 16, 8 or 4 bits, and attention over it.  Thin
Python binding of the C ABI in ``include/sage_kv.h``; every step runs in the
CUDA kernels of ``_build/libsagefp4.so``, there is no fallback, and a failed
call raises.

``append`` stores new keys and values, ``attention`` lets new tokens' queries
attend to their sequences' cached tokens (prompts, chunks and single tokens
alike, grouped query heads), ``read`` hands sequences back as the dense bf16
tensors that ``sage_fp4.attention`` takes.  All three take the same batch
tensors, int32 on the GPU: ``cu_q`` [B + 1] (the packed rows of each
sequence's new tokens), ``kv_len`` [B] (its cached tokens, the new ones among
them) and ``block_table`` [B, pages].  They never look at these on the host, so
a captured call follows changing lengths.  No gradients flow through them.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

from . import sage_fp4 as _fp4
from .sage_fp4 import EINVAL, SageFp4Error, sage_fp4_strides

_HEADER = os.path.join(os.path.dirname(_fp4._HEADER), "sage_kv.h")
INT32_MAX = 0x7fffffff
FORMATS = {"bf16": 0, "e4m3": 1, "nvfp4": 2}  # SAGE_KV_*
_lock = threading.Lock()
_declared = set()


class sage_kv_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales", "status")]
    _fields_ += [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "H", "D", "format")]


class sage_kv_batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("cu_q", "kv_len", "block_table")]
    _fields_ += [("table_stride", ctypes.c_int64), ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class sage_kv_rows(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int64), ("h", ctypes.c_int64)]


def header_functions() -> list:
    """Names of the functions declared in include/sage_kv.h."""
    text = open(_HEADER).read()
    return sorted(set(re.findall(r"^[a-z_ 0-9\*]+?\b(sage_kv_[a-z_0-9]+)\s*\(", text, re.M)))


def lib() -> ctypes.CDLL:
    L = _fp4.load()
    if id(L) not in _declared:
        with _lock:
            vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
            cp, bp, sp = (ctypes.POINTER(s) for s in (sage_kv_cache, sage_kv_batch, sage_fp4_strides))
            rows = sage_kv_rows
            sig = {
                "sage_kv_append": (i, [cp, bp, vp, rows, vp, rows, i, vp]),
                "sage_kv_read": (i, [cp, bp, vp, sp, vp, sp, i, vp]),
                "sage_kv_attn_workspace_bytes": (sz, [cp, i, i, i]),
                "sage_kv_attn": (i, [cp, bp, vp, rows, vp, rows, vp, i, i, i, i, f, vp, sz, vp]),
                "sage_kv_attn_stall_test": (i, [cp, bp, vp, rows, vp, rows, i, i, ctypes.c_uint64, vp, sz, vp]),
                "sage_kv_get_status": (i, [cp, vp]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype, fn.argtypes = res, args
            _declared.add(id(L))
    return L


# ------------------------------------------------------------- raw entry points
def sage_kv_append(cache, batch, k_ptr, k_rows, v_ptr, v_rows, T: int, stream) -> int:
    return lib().sage_kv_append(cache, batch, k_ptr, k_rows, v_ptr, v_rows, T, stream)


def sage_kv_read(cache, batch, k_ptr, k_strides, v_ptr, v_strides, N: int, stream) -> int:
    """Strides: sage_fp4_strides or None (contiguous [B, H, N, D])."""
    return lib().sage_kv_read(cache, batch, k_ptr, k_strides, v_ptr, v_strides, N, stream)


def sage_kv_attn_workspace_bytes(cache, B: int, T: int, Hq: int) -> int:
    return lib().sage_kv_attn_workspace_bytes(cache, B, T, Hq)


def sage_kv_attn(cache, batch, q_ptr, q_rows, o_ptr, o_rows, lse_ptr, T: int, Hq: int, causal, window: int, scale: float,
                 ws_ptr, ws_bytes: int, stream) -> int:
    return lib().sage_kv_attn(cache, batch, q_ptr, q_rows, o_ptr, o_rows, lse_ptr, T, Hq, int(causal), window, scale,
                              ws_ptr, ws_bytes, stream)


def sage_kv_attn_stall_test(cache, batch, q_ptr, q_rows, o_ptr, o_rows, T: int, Hq: int, wait_limit_ns: int, ws_ptr,
                            ws_bytes: int, stream) -> int:
    return lib().sage_kv_attn_stall_test(cache, batch, q_ptr, q_rows, o_ptr, o_rows, T, Hq, wait_limit_ns, ws_ptr, ws_bytes,
                                         stream)


def sage_kv_get_status(cache, stream) -> int:
    return lib().sage_kv_get_status(cache, stream)


# ------------------------------------------------------------- torch conveniences
def _fmt(fmt: str) -> int:
    if fmt not in FORMATS:
        raise SageFp4Error(EINVAL, f"format must be one of {tuple(FORMATS)}, not {fmt!r}")
    return FORMATS[fmt]


def _parts(fmt: str, num_pages: int, page_size: int, H: int, D: int):
    """(shape, torch dtype) of the codes and of the scales (None for bf16)."""
    import torch
    lead = (num_pages, H, page_size)
    if fmt == "bf16":
        return (lead + (D,), torch.bfloat16), None
    if fmt == "e4m3":
        return (lead + (D,), torch.uint8), (lead, torch.uint8)
    return (lead + (D // 2,), torch.uint8), (lead + (D // 16,), torch.uint8)


class PagedCache:
    """Pages of keys and values of H heads of D channels.

    fmt: "bf16", "e4m3" (E4M3 codes with a power-of-two scale per row) or
    "nvfp4" (E2M1 codes with an E4M3 scale per 16 channels).  The buffers are
    the attributes k_codes, v_codes, k_scales, v_scales (layouts in
    include/sage_kv.h).  A new cache's contents are undefined until written."""

    def __init__(self, num_pages: int, page_size: int, H: int, D: int, fmt: str = "bf16", device=None):
        import torch
        _fmt(fmt)
        if num_pages < 0 or H < 1 or D not in (64, 128):
            raise SageFp4Error(EINVAL, f"cache of {num_pages} pages, H={H}, D={D}")
        codes, scales = _parts(fmt, num_pages, page_size, H, D)
        new = lambda part: part and torch.empty(part[0], dtype=part[1], device=device or "cuda")  # noqa: E731
        self._take(new(codes), new(codes), new(scales), new(scales), fmt, D)

    @classmethod
    def wrap(cls, k_codes, v_codes, k_scales=None, v_scales=None, fmt: str = "bf16"):
        """A cache over buffers that the caller holds (their layouts are those
        of the attributes; nothing is copied)."""
        self = cls.__new__(cls)
        _fmt(fmt)
        if k_codes.dim() != 4:
            raise SageFp4Error(EINVAL, "k_codes must be [pages, H, page_size, row]")
        self._take(k_codes, v_codes, k_scales, v_scales, fmt, k_codes.shape[3] * (2 if fmt == "nvfp4" else 1))
        return self

    def _take(self, k_codes, v_codes, k_scales, v_scales, fmt, D):
        import torch
        self.fmt, self.D = fmt, D
        self.num_pages, self.H, self.page_size = k_codes.shape[:3]
        ps = self.page_size
        if D not in (64, 128) or self.H < 1 or ps < 16 or ps > 1024 or ps & (ps - 1):
            raise SageFp4Error(EINVAL, f"cache of H={self.H}, D={D}, pages of {ps} tokens (a power of two from 16 to 1024)")
        codes, scales = _parts(fmt, self.num_pages, ps, self.H, D)
        for x, want, nm in ((k_codes, codes, "k_codes"), (v_codes, codes, "v_codes"), (k_scales, scales, "k_scales"),
                            (v_scales, scales, "v_scales")):
            if want is None:
                if x is not None:
                    raise SageFp4Error(EINVAL, f"{nm} given for a bf16 cache")
            elif x is None or not x.is_cuda or x.dtype != want[1] or tuple(x.shape) != want[0] or \
                    not x.is_contiguous() or x.device != k_codes.device:
                raise SageFp4Error(EINVAL, f"{nm} must be a contiguous {want[1]} CUDA tensor {want[0]} on one device")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.device, self.index = k_codes.device, k_codes.get_device()
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        ptr = lambda x: None if x is None else x.data_ptr()  # noqa: E731
        self.struct = sage_kv_cache(ptr(k_codes), ptr(v_codes), ptr(k_scales), ptr(v_scales), ptr(self.status),
                                    self.num_pages, ps, self.H, D, FORMATS[fmt])
        self.buffers = [x for x in (k_codes, v_codes, k_scales, v_scales, self.status) if x is not None]
        self._bytes = {}  # workspace sizes asked for last

    def get_status(self, stream=None) -> int:
        """Synchronise, return the status word (EINDEX, ETIMEOUT) and reset it to 0."""
        import torch
        with torch.cuda.device(self.device):
            return sage_kv_get_status(self.struct, _fp4._stream(stream))


def _batch(cache: PagedCache, cu_q, kv_len, block_table) -> sage_kv_batch:
    import torch
    ks, ts, dev = kv_len.shape, block_table.shape, cache.index
    B = ks[0] if len(ks) == 1 else -1
    for x, nm in ((cu_q, "cu_q"), (kv_len, "kv_len"), (block_table, "block_table")):
        if x is not None and (x.dtype != torch.int32 or x.get_device() != dev):
            raise SageFp4Error(EINVAL, f"{nm} must be an int32 tensor on the cache's device")
    if B < 0 or not kv_len.is_contiguous() or (cu_q is not None and (cu_q.shape != (B + 1,) or not cu_q.is_contiguous())):
        raise SageFp4Error(EINVAL, "kv_len must be a contiguous [B], cu_q a contiguous [B + 1] tensor")
    if len(ts) != 2 or ts[0] != B or max(B, ts[1]) > INT32_MAX:
        raise SageFp4Error(EINVAL, f"block_table must be [{B}, pages], both below 2^31")
    pages, (row, one) = ts[1], block_table.stride()
    if (pages > 1 and one != 1) or (B > 1 and row < pages):
        raise SageFp4Error(EINVAL, "block_table must have a contiguous last axis and rows of their own")
    return sage_kv_batch(None if cu_q is None else cu_q.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
                         row if B > 1 else pages, B, pages)


def _rows(x, cache: PagedCache, name: str, H: int | None = None):
    """Rows, heads, and the token and head strides of a packed bf16 [T, H, D] tensor."""
    import torch
    shape, stride = x.shape, x.stride()
    if x.dtype != torch.bfloat16 or x.get_device() != cache.index or len(shape) != 3 or shape[2] != cache.D or \
            (stride[2] != 1 and x.numel()):
        raise SageFp4Error(EINVAL, f"{name} must be a bf16 tensor [T, heads, {cache.D}] on the cache's device with a "
                                   "contiguous last axis")
    t, h, _ = shape
    if max(t, h) > INT32_MAX:  # a broadcast tensor; ctypes would cut the numbers
        raise SageFp4Error(EINVAL, f"{name} has {t} rows of {h} heads, more than 2^31 - 1")
    if H is not None and h != H:
        raise SageFp4Error(EINVAL, f"{name} has {h} heads, not {H}")
    return t, h, sage_kv_rows(stride[0] if t > 1 else 0, stride[1] if h > 1 else 0)


def append(cache: PagedCache, k, v, cu_q, kv_len, block_table, stream=None) -> None:
    """Store the new tokens' keys and values, bf16 [T, H, D] (any strides with a
    contiguous last axis and 16-byte aligned rows), quantized to the cache's
    format.  Rows cu_q[b] .. cu_q[b + 1] - 1 become the last tokens of
    sequence b, whose length kv_len[b] counts them already."""
    batch = _batch(cache, cu_q, kv_len, block_table)
    (T, _, kr), (Tv, _, vr) = _rows(k, cache, "k", cache.H), _rows(v, cache, "v", cache.H)
    if T != Tv:
        raise SageFp4Error(EINVAL, f"k has {T} rows, v {Tv}")
    _fp4._call(lib().sage_kv_append, "sage_kv_append", cache.index, stream,
               None if stream is None else (k, v, cu_q, kv_len, block_table, *cache.buffers), cache.struct, batch, k.data_ptr(), kr, v.data_ptr(), vr, T)


def read(cache: PagedCache, kv_len, block_table, N: int, layout: str = "HND", out=None, stream=None):
    """The first N tokens of every sequence as dense bf16 (k, v) in `layout`
    ("HND" = [B, H, N, D], "NHD" = [B, N, H, D]); tokens past a sequence's
    length are zeros.  out: (k, v) to write instead of new tensors, of memory of
    their own."""
    import torch
    batch = _batch(cache, None, kv_len, block_table)
    if layout not in _fp4.LAYOUTS or not 0 <= N <= INT32_MAX:
        raise SageFp4Error(EINVAL, f"layout must be one of {_fp4.LAYOUTS}, not {layout!r}; N = {N}")
    B, H, D = batch.B, cache.H, cache.D
    shape = (B, H, N, D) if layout == "HND" else (B, N, H, D)
    if out is None:
        k, v = (torch.empty(shape, dtype=torch.bfloat16, device=cache.device) for _ in range(2))
    else:
        k, v = out
    strides = []
    for x, nm in ((k, "k"), (v, "v")):
        if out is None and layout == "HND":  # contiguous, as the C ABI takes it without strides
            strides.append(None)
            continue
        if x.dtype != torch.bfloat16 or x.get_device() != cache.index or tuple(x.shape) != shape or (x.stride(3) != 1 and x.numel()):
            raise SageFp4Error(EINVAL, f"{nm} must be a bf16 tensor {shape} on the cache's device with a contiguous last axis")
        _fp4._own_elements(x, nm)
        s = [st if n > 1 else 0 for st, n in zip(x.stride(), shape)]
        strides.append(sage_fp4_strides(s[0], s[1], s[2]) if layout == "HND" else sage_fp4_strides(s[0], s[2], s[1]))
    if out is not None and k.data_ptr() == v.data_ptr() and k.numel():
        raise SageFp4Error(EINVAL, "out: k and v share memory")
    _fp4._call(lib().sage_kv_read, "sage_kv_read", cache.index, stream,
               None if stream is None else (k, v, kv_len, block_table, *cache.buffers),
               cache.struct, batch, k.data_ptr(), strides[0], v.data_ptr(), strides[1], N)
    return k, v


def attention_workspace_bytes(cache: PagedCache, B: int, T: int, Hq: int) -> int:
    """Bytes of the workspace that ``attention`` takes for these sizes."""
    n = cache._bytes.get((B, T, Hq))
    if n is None:
        n = sage_kv_attn_workspace_bytes(cache.struct, B, T, Hq)
        if n == 0:
            raise SageFp4Error(EINVAL, f"B={B}, T={T}, Hq={Hq} over a cache of {cache.H} heads")
        if len(cache._bytes) >= 64:
            cache._bytes.clear()
        cache._bytes[B, T, Hq] = n
    return n


def attention(q, cache: PagedCache, cu_q, kv_len, block_table, causal: bool = True, scale=None, window: int | None = None,
              out=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of new tokens over the cache: q bf16 [T, Hq, D] (any strides
    with a contiguous last axis and 16-byte aligned rows; Hq a multiple of the
    cache's heads) -> o bf16 [T, Hq, D].

    causal: a new token sees the tokens up to its own position (it is one of
    the last of kv_len[b]); False: all kv_len[b] (cross attention).  window:
    only the last `window` of those.  scale: softmax scale (default
    1/sqrt(D)).  A row that sees nothing is zeros; rows behind cu_q[B] are
    left as they were.  out: a tensor to write, which shares no memory with q or
    the cache.  return_lse: also the natural-log log-sum-exp, float32
    [T, Hq] (-inf for a row that sees nothing).  workspace: uint8 tensor of
    attention_workspace_bytes (a temporary one by default); calls sharing one
    must be ordered.

    One kernel serves a call, by its average of new tokens a sequence: single
    tokens and long chunks are faster in a call each."""
    import torch
    batch = _batch(cache, cu_q, kv_len, block_table)
    T, Hq, qr = _rows(q, cache, "q")
    if Hq < 1 or Hq % cache.H:
        raise SageFp4Error(EINVAL, f"{Hq} query heads over {cache.H} key/value heads")
    if window is not None and not 1 <= window <= INT32_MAX:
        raise SageFp4Error(EINVAL, f"window must be from 1 to 2^31 - 1, not {window}")
    if out is None:
        out = torch.empty((T, Hq, cache.D), dtype=torch.bfloat16, device=cache.device)
        orow = sage_kv_rows(Hq * cache.D, cache.D)
    else:
        To, _, orow = _rows(out, cache, "out", Hq)
        _fp4._own_elements(out, "out")
        if To != T:
            raise SageFp4Error(EINVAL, f"out has {To} rows, q {T}")
        if T and out.data_ptr() == q.data_ptr():
            raise SageFp4Error(EINVAL, "out shares memory with q")  # parts of a row are still to be read
    lse = torch.empty((T, Hq), dtype=torch.float32, device=cache.device) if return_lse else None
    nbytes = attention_workspace_bytes(cache, batch.B, T, Hq)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    elif workspace.dtype != torch.uint8 or workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise SageFp4Error(EINVAL, "workspace must be a contiguous uint8 tensor on the cache's device")
    else:
        nbytes = workspace.numel()
    _fp4._call(lib().sage_kv_attn, "sage_kv_attn", cache.index, stream,
               None if stream is None else (q, out, lse, workspace, cu_q, kv_len, block_table, *cache.buffers), cache.struct, batch, q.data_ptr(), qr,
               out.data_ptr(), orow, None if lse is None else lse.data_ptr(), T, Hq, bool(causal), window or 0,
               cache.D ** -0.5 if scale is None else float(scale), workspace.data_ptr(), nbytes)
    return (out, lse) if return_lse else out
