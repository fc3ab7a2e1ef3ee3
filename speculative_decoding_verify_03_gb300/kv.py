"""The key/value cache of the verify step and the attention that reads it:
the binding of include/spec_kv.h."""
from __future__ import annotations

import ctypes

import torch

SPEC_KV_BF16, SPEC_KV_E4M3 = 0, 1
ROW_BAD_LENGTH, ROW_BAD_PAGE = 1 << 7, 1 << 8

_i32, _f32, _bf16 = torch.int32, torch.float32, torch.bfloat16
_byref = ctypes.byref


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# torch's own short ways to the same address and number, where it has them (2 us a call less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class SpecKvCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class SpecKvBatch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("gamma_max", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
                ("table_row_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("prefix_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("gamma_per_row", ctypes.c_void_p)]


_Strides = ctypes.c_int64 * 3


class KVCache:
    """A paged cache on the GPU: k_pages and v_pages [n_pages, n_kv_heads,
    page_size, head_dim], bfloat16, or float8_e4m3fn with k_exp and v_exp
    [n_pages, n_kv_heads, page_size] int8 (a stored y stands for y * 2^e).
    Pages may be strided (both halves of one allocation, say); what is inside
    a page is contiguous.  The tensors are the caller's: the cache keeps them
    alive and describes them to the library."""

    def __init__(self, k_pages, v_pages, k_exp=None, v_exp=None):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must be [n_pages, n_kv_heads, page_size, head_dim]")
        if k_pages.dtype != v_pages.dtype or k_pages.dtype not in (torch.bfloat16,
                                                                   torch.float8_e4m3fn):
            raise TypeError("pages must be bfloat16 or float8_e4m3fn")
        n, H, S, D = k_pages.shape
        if n and not (k_pages[0].is_contiguous() and v_pages[0].is_contiguous()):
            raise ValueError("the inside of a page must be contiguous")
        if k_pages.dtype == torch.float8_e4m3fn:
            for t in (k_exp, v_exp):
                if t is None or t.dtype != torch.int8:
                    raise TypeError("an e4m3 cache needs int8 k_exp and v_exp")
                if t.shape != (n, H, S) or not t.is_contiguous():
                    raise ValueError("k_exp and v_exp must be contiguous [n_pages, n_kv_heads, page_size]")
            fmt = SPEC_KV_E4M3
        else:
            if k_exp is not None or v_exp is not None:
                raise ValueError("a bfloat16 cache has no exponents")
            fmt = SPEC_KV_BF16
        for t in (v_pages, k_exp, v_exp):
            if t is not None and t.device != k_pages.device:
                raise ValueError("the cache's tensors must be on one device")
        self.k_pages, self.v_pages, self.k_exp, self.v_exp = k_pages, v_pages, k_exp, v_exp
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n, H, S, D
        self.device = k_pages.device
        ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        self.struct = SpecKvCache(ptr(k_pages), ptr(v_pages), ptr(k_exp), ptr(v_exp),
                                  k_pages.stride(0) if n else H * S * D,
                                  v_pages.stride(0) if n else H * S * D, n, S, H, D, fmt)
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, n_pages, n_kv_heads, page_size, head_dim, dtype=None, device="cuda"):
        """A cache of new pages; dtype float8_e4m3fn (the default) or bfloat16."""
        dtype = dtype or torch.float8_e4m3fn
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype == torch.bfloat16:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.int8, device=device) for _ in range(2)))




def _int32(name, t, n, device):
    """A contiguous int32 vector of n elements on the cache's device."""
    if t.dtype != _i32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 1 or t.shape[0] != n or t.device != device:
        raise ValueError(f"{name} must be [{n}] on {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _batch(cache, page_table, kv_len, gamma_max, prefix_table, prefix_len, gamma_per_row):
    dev = cache.device
    B = kv_len.shape[0] if kv_len.dim() == 1 else -1
    len_ptr = _int32("kv_len", kv_len, B, dev)
    if page_table.dtype != _i32:
        raise TypeError("page_table must be int32")
    shape = page_table.shape
    if len(shape) != 2 or shape[0] != B or page_table.device != dev:
        raise ValueError(f"page_table must be [{B}, max_pages] on {dev}")
    mp = shape[1]
    row, col = page_table.stride()
    if col != 1 and B and mp:
        raise ValueError("page_table rows must be contiguous")
    gamma = None if gamma_per_row is None else _int32("gamma_per_row", gamma_per_row, B, dev)
    pt, prefix_len = None, int(prefix_len)
    if prefix_len > 0:
        need = -(-prefix_len // cache.page_size)
        if prefix_table is None or prefix_table.dim() != 1 or prefix_table.shape[0] < need:
            raise ValueError(f"prefix_table must hold the prefix's {need} page ids")
        pt = _int32("prefix_table", prefix_table, prefix_table.shape[0], dev)
    return SpecKvBatch(B, gamma_max, mp, prefix_len, row if B > 1 else mp, page_table.data_ptr(), pt, len_ptr, gamma)


_library = None


def _lib():
    """The loaded library, looked up once."""
    global _library
    if _library is None:
        from . import lib
        _library = lib()
    return _library


def _check(code):
    if code != 0:
        from . import _check as check
        check(code)


def _elsewhere(stream, device):
    """Whether a call has to go to another stream or device than the current ones."""
    return stream is not None or device.type != "cuda" or device.index != _device()


def _on(stream, device, call, *args):
    """call(*args) with the device and the stream (if given) current: kernels run on
    the current device, and what the call allocates is to be the stream's.  What it
    returns may be freed by its caller while the caller's own stream still uses
    it: the allocator is told."""
    if device.type != "cuda":
        from . import SpecError
        raise SpecError(f"the cache is on {device}: this library has no CPU path")
    if stream is None:
        with torch.cuda.device(device):
            return call(*args)
    if stream.device != device:
        raise ValueError(f"the stream must be on {device}")
    with torch.cuda.stream(stream):
        got = call(*args)
    here = torch.cuda.current_stream(device)
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            t.record_stream(here)
    return got


def _status(with_status, B, device):
    return torch.empty(B, dtype=_i32, device=device) if with_status else None


def _ptr(t):
    return t.data_ptr() if t is not None else None


def spec_kv_append(cache, k, v, page_table, kv_len, gamma_per_row=None, prefix_len=0,
                   with_status=False, stream=None):
    """Append a step's keys and values to the cache (see spec_kv_append in
    include/spec_kv.h): k and v [B, n, n_kv_heads, head_dim] float32 or
    bfloat16 (any strides, contiguous head_dim), token t of sequence b to
    position kv_len[b] + t; with gamma_per_row [B] int32, sequence b has
    gamma_b + 1 tokens.  page_table [B, max_pages] int32 holds the sequences'
    own pages, whose first position is prefix_len.  stream: as a call within
    torch.cuda.stream(stream); what it returns may be used on the caller's
    stream as well, once that waits for it.  Updates the cache in
    place; returns row_status [B] when with_status, else None."""
    dev = cache.device
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4 or v.shape != shape or v.dtype != dtype:
        raise ValueError("k and v must be [B, n, n_kv_heads, head_dim] of one dtype")
    B, n, H, D = shape
    if H != cache.n_kv_heads or D != cache.head_dim or B != kv_len.shape[0] or n < 1:
        raise ValueError("k and v do not match the cache's heads or kv_len's rows")
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError(f"k and v must be float32 or bfloat16, got {dtype}")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on {dev}")
    ks, vs = k.stride(), v.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the head_dim axis must be contiguous")
    b = _batch(cache, page_table, kv_len, n - 1, None, 0, gamma_per_row)
    if _elsewhere(stream, dev):
        return _on(stream, dev, spec_kv_append, cache, k, v, page_table, kv_len, gamma_per_row, prefix_len, with_status)
    if prefix_len:
        b.prefix_len = int(prefix_len)
        b.prefix_table = b.page_table  # not read: the step is past the prefix
    st = _status(with_status, B, dev)
    code = _lib().spec_kv_append(cache.ref, _byref(b), k.data_ptr(), v.data_ptr(), 0 if dtype is _f32 else 1,
                                 _byref(_Strides(*ks[:3])), _byref(_Strides(*vs[:3])), _ptr(st),
                                 _raw_stream(dev.index))
    if code:
        _check(code)
    return st


def spec_kv_read(cache, page_table, kv_len, n, begin=0, prefix_table=None, prefix_len=0,
                 dtype=None, with_status=False, stream=None):
    """Read positions begin .. begin + n - 1 of every sequence back (see
    spec_kv_read in include/spec_kv.h): returns (k, v) [B, n, n_kv_heads,
    head_dim] in dtype (bfloat16 by default, or float32), zeros from kv_len[b]
    on, and row_status [B] when with_status.  stream: as a call within
    torch.cuda.stream(stream); what it returns may be used on the caller's
    stream as well, once that waits for it."""
    dev = cache.device
    dtype = dtype or _bf16
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError("dtype must be bfloat16 or float32")
    if n < 0 or begin < 0:
        raise ValueError("begin and n must not be negative")
    b = _batch(cache, page_table, kv_len, 0, prefix_table, prefix_len, None)
    if _elsewhere(stream, dev):
        return _on(stream, dev, spec_kv_read, cache, page_table, kv_len, n, begin, prefix_table, prefix_len, dtype,
                   with_status)
    n, begin = int(n), int(begin)
    shape = (b.B, n, cache.n_kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=dtype, device=dev)
    v = torch.empty(shape, dtype=dtype, device=dev)
    st = _status(with_status, b.B, dev)
    code = _lib().spec_kv_read(cache.ref, _byref(b), begin, n, 0 if dtype is _f32 else 1, k.data_ptr(), v.data_ptr(),
                               _ptr(st), _raw_stream(dev.index))
    if code:
        _check(code)
    return (k, v, st) if with_status else (k, v)


def attend_workspace_bytes(cache, batch, n_heads) -> int:
    """Workspace bytes of spec_attend for these shapes: of the SpecKvBatch, B,
    gamma_max, max_pages (the page table's columns) and prefix_len count."""
    shapes = SpecKvBatch(batch.B, batch.gamma_max, batch.max_pages, batch.prefix_len, batch.max_pages)
    return _lib().spec_attend_workspace_size(cache.ref, _byref(shapes), n_heads)


def spec_attend(q, cache, page_table, kv_len, prefix_table=None, prefix_len=0, gamma_per_row=None,
                scale=None, workspace="auto", out=None, with_status=False, stream=None):
    """The verify step's attention (see spec_attend in include/spec_kv.h): q
    [B, gamma_max + 1, n_heads, head_dim] bfloat16 (any strides, contiguous
    head_dim); query i of sequence b attends to positions 0 .. kv_len[b] + i,
    the first prefix_len of them in the shared pages prefix_table, the others
    in the sequence's own pages page_table[b].  The step's keys and values are
    in the cache already.  scale defaults to head_dim ** -0.5.  workspace:
    "auto" (the call's own, from torch's allocator: calls from several threads
    and in captured graphs do not share it) or a uint8 CUDA tensor of
    attend_workspace_bytes, which no other call may use meanwhile.  out: a pair
    of contiguous tensors for the results, or None.  stream: as a call within
    torch.cuda.stream(stream); what it returns may be used on the caller's
    stream as well, once that waits for it.  Returns (out [B, gamma_max + 1,
    n_heads, head_dim] bfloat16, lse [B, gamma_max + 1, n_heads] float32), and
    row_status [B] when with_status."""
    dev = cache.device
    shape = q.shape
    if q.dtype is not _bf16:
        raise TypeError("q must be bfloat16")
    if len(shape) != 4 or shape[0] != kv_len.shape[0] or shape[1] < 1 or shape[3] != cache.head_dim:
        raise ValueError("q must be [B, gamma_max + 1, n_heads, head_dim]")
    if q.device != dev:
        raise ValueError(f"q must be on {dev}")
    qs = q.stride()
    if qs[3] != 1:
        raise ValueError("the head_dim axis must be contiguous")
    B, N, Hq, D = shape
    if Hq < 1 or Hq % cache.n_kv_heads:
        raise ValueError("n_heads must be a multiple of the cache's n_kv_heads")
    b = _batch(cache, page_table, kv_len, N - 1, prefix_table, prefix_len, gamma_per_row)
    if _elsewhere(stream, dev):
        return _on(stream, dev, spec_attend, q, cache, page_table, kv_len, prefix_table, prefix_len, gamma_per_row,
                   scale, workspace, out, with_status)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a tensor")
        workspace = torch.empty(_lib().spec_attend_workspace_size(cache.ref, _byref(b), Hq), dtype=torch.uint8, device=dev)
    elif workspace is None or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be 'auto' or a contiguous tensor on {dev}")
    if out is None:
        o = torch.empty(shape, dtype=_bf16, device=dev)
        lse = torch.empty(shape[:3], dtype=_f32, device=dev)
    else:
        o, lse = out
        if (o.shape != shape or o.dtype is not _bf16 or not o.is_contiguous() or lse.shape != shape[:3] or
                lse.dtype is not _f32 or not lse.is_contiguous() or o.device != dev or lse.device != dev):
            raise ValueError("out must be contiguous bfloat16 and float32 tensors of the results' shapes")
    st = _status(with_status, B, dev)
    code = _lib().spec_attend(cache.ref, _byref(b), q.data_ptr(), Hq, _byref(_Strides(*qs[:3])),
                              D ** -0.5 if scale is None else float(scale), o.data_ptr(), lse.data_ptr(), _ptr(st),
                              workspace.data_ptr(), workspace.numel() * workspace.element_size(), _raw_stream(dev.index))
    if code:
        _check(code)
    return (o, lse, st) if with_status else (o, lse)
