"""split_kv_gb300 -- split-KV decode attention (Flash-Decoding) for GB300.

A thin ctypes binding over the C ABI of ``lib/libfd.so`` (declared in
``include/fd.h``).  Every function has the C name and does argument
marshalling only: torch tensors are passed as device pointers, streams as
``cudaStream_t`` handles, and every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback: if the library is missing
the first call raises.

Typical use::

    import split_kv_gb300 as fd
    desc = fd.make_desc(q, k_cache, v_cache, max_seqlen=int(seqlens_host.max()))
    desc.n_splits = fd.fd_plan(B, Hq, Hkv, 128, seqlens_host)
    ws = torch.empty(fd.fd_workspace_size(desc, desc.n_splits), dtype=torch.uint8, device="cuda")
    fd.check(fd.fd_decode(desc, q, k_cache, v_cache, seqlens, None, out, lse, ws))
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import _build

FD_OK = 0
FD_ERR_INVALID_ARG = -1
FD_ERR_UNSUPPORTED = -2
FD_ERR_WORKSPACE = -3
FD_ERR_CUDA = -4
FD_ERR_DEVICE_TIMEOUT = -5
FD_ERR_DEVICE_BOUNDS = -6

FD_F16, FD_BF16, FD_F32, FD_E4M3 = 0, 1, 2, 3
FD_MAX_SPLITS = 128
FD_TILE_TOKENS = 128
FD_STATIC_WORKSPACE_BYTES = 8 << 20
FD_FLAG_CUDA_CORES = 1
FD_FLAG_TEST_DROP_FIRST_STAGE = 1 << 16

LIB_PATH = _build.LIB_PATH

# every function the header declares (checked against include/fd.h by the tests)
EXPORTS = ("fd_abi_version", "fd_status_string", "fd_num_sms", "fd_plan_splits", "fd_plan",
           "fd_plan_desc", "fd_workspace_size", "fd_decode", "fd_split_states", "fd_combine_states",
           "fd_device_status", "fd_decode_status", "fd_decode_static", "fd_decode_scaled",
           "fd_cache_store", "fd_page_tables", "fd_prompt", "fd_prompt_workspace_size")


class FdDesc(ctypes.Structure):
    """Mirror of ``fd_desc`` (include/fd.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("q_stride_b", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("k_stride_b", ctypes.c_int64), ("k_stride_h", ctypes.c_int64), ("k_stride_t", ctypes.c_int64),
        ("v_stride_b", ctypes.c_int64), ("v_stride_h", ctypes.c_int64), ("v_stride_t", ctypes.c_int64),
        ("kv_extent", ctypes.c_int64),
        ("page_size", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("max_seqlen", ctypes.c_int32), ("n_splits", ctypes.c_int32),
        ("flags", ctypes.c_int32), ("q_len", ctypes.c_int32),
        ("q_stride_t", ctypes.c_int64),
        ("q_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
    ]

    def copy(self) -> "FdDesc":
        d = FdDesc()
        ctypes.pointer(d)[0] = self
        return d


class FdKvScales(ctypes.Structure):
    """Mirror of ``fd_kv_scales`` (include/fd.h)."""
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_stride_b", ctypes.c_int64), ("k_stride_h", ctypes.c_int64), ("k_stride_n", ctypes.c_int64),
        ("v_stride_b", ctypes.c_int64), ("v_stride_h", ctypes.c_int64), ("v_stride_n", ctypes.c_int64),
        ("block", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]
    shape = None    # (leading, KV heads, blocks) of the tensors, by make_scales


class FdStoreDesc(ctypes.Structure):
    """Mirror of ``fd_store_desc`` (include/fd.h)."""
    _fields_ = [
        ("n_tokens", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("src_dtype", ctypes.c_int32),
        ("k_src_stride_t", ctypes.c_int64), ("k_src_stride_h", ctypes.c_int64),
        ("v_src_stride_t", ctypes.c_int64), ("v_src_stride_h", ctypes.c_int64),
        ("k_stride_b", ctypes.c_int64), ("k_stride_h", ctypes.c_int64), ("k_stride_t", ctypes.c_int64),
        ("v_stride_b", ctypes.c_int64), ("v_stride_h", ctypes.c_int64), ("v_stride_t", ctypes.c_int64),
        ("kv_extent", ctypes.c_int64), ("page_size", ctypes.c_int32), ("batch", ctypes.c_int32),
    ]


class FdPageDesc(ctypes.Structure):
    """Mirror of ``fd_page_desc`` (include/fd.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "page_size", "max_pages_per_seq", "n_pages",
                                              "n_free_max", "n_slots")]


class FdPromptDesc(ctypes.Structure):
    """Mirror of ``fd_prompt_desc`` (include/fd.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("k_stride_t", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
        ("v_stride_t", ctypes.c_int64), ("v_stride_h", ctypes.c_int64),
        ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
        ("max_q", ctypes.c_int32), ("max_k", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("n_splits", ctypes.c_int32),
        ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class FdError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        super().__init__(f"{what}: {fd_status_string(status)} ({status})" if what
                         else f"{fd_status_string(status)} ({status})")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() "
                               "(the decode path has no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        dp = ctypes.POINTER(FdDesc)
        sig = {
            "fd_abi_version": (i32, []),
            "fd_status_string": (ctypes.c_char_p, [i32]),
            "fd_num_sms": (i32, [i32]),
            "fd_plan_splits": (i32, [i64, i64, i64, i32]),
            "fd_plan": (i32, [i32, i32, i32, i32, vp, vp, i32, i32, i32]),
            "fd_plan_desc": (i32, [dp, vp, i32]),
            "fd_workspace_size": (sz, [dp, i32]),
            "fd_decode": (i32, [dp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "fd_split_states": (i32, [dp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "fd_combine_states": (i32, [dp, vp, sz, vp, vp, vp]),
            "fd_device_status": (i32, [vp, i32]),
            "fd_decode_status": (i32, [vp]),
            "fd_decode_static": (i32, [dp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "fd_decode_scaled": (i32, [dp, ctypes.POINTER(FdKvScales), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "fd_cache_store": (i32, [ctypes.POINTER(FdStoreDesc), ctypes.POINTER(FdKvScales),
                                     vp, vp, vp, vp, vp, vp]),
            "fd_page_tables": (i32, [ctypes.POINTER(FdPageDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "fd_prompt_workspace_size": (sz, [ctypes.POINTER(FdPromptDesc)]),
            "fd_prompt": (i32, [ctypes.POINTER(FdPromptDesc), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
        return lib


def _ptr(x):
    """Device/host address of a torch tensor, an int address, or None."""
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:
        if isinstance(x, int):
            return x
        raise TypeError(f"cannot take the address of {type(x)}") from None


_raw_stream = None


def _current_stream() -> int:
    """Handle of torch's current stream on the current device (the raw query
    costs 0.2 us a call, building torch's Stream object 2.9)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        torch.cuda.current_stream()                # (initialises CUDA)
        if get is None or device is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream
        else:
            _raw_stream = lambda: get(device())
    return _raw_stream()


def _stream(s):
    if s is None:
        return _raw_stream() if _raw_stream is not None else _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _nbytes(x) -> int:
    return 0 if x is None else x.nbytes


def _check_out(out, lse, out_dtype: int, rows: int) -> None:
    """The tensors that a call writes are as large as its descriptor says (addresses go unchecked)."""
    try:
        size = 4 if out_dtype == FD_F32 else 2
        if out.element_size() != size or out.nbytes < rows * size * 128 or not out.is_contiguous():
            raise ValueError(f"out must be contiguous, of the descriptor's out_dtype, with {rows} rows")
    except AttributeError:
        pass
    if lse is not None:
        try:
            if lse.nbytes < 4 * rows or lse.element_size() != 4 or not lse.is_contiguous():
                raise ValueError(f"lse must be {rows} contiguous float32")
        except AttributeError:
            pass


def _check_scales(desc, scales: FdKvScales) -> None:
    """make_scales' tensors cover the cache of a decode or store descriptor (the C ABI sees no extents)."""
    if scales.shape is None:
        return
    lead, heads, blocks = scales.shape
    page = desc.page_size
    tokens = page if page > 0 else desc.kv_extent
    if lead < (desc.kv_extent if page > 0 else desc.batch) or heads < desc.n_kv_heads or blocks * scales.block < tokens:
        raise ValueError(f"scales {scales.shape} of {scales.block}-token blocks do not cover the cache")


def check(status: int, what: str = "") -> int:
    if int(status) < 0:
        raise FdError(status, what)
    return int(status)


# ---------------------------------------------------------------- C ABI
def fd_abi_version() -> int:
    return int(_load().fd_abi_version())


def fd_status_string(status: int) -> str:
    return _load().fd_status_string(int(status)).decode()


def fd_num_sms(device: int = -1) -> int:
    return int(_load().fd_num_sms(int(device)))


def fd_plan_splits(work_items: int, slots: int, n_kv_blocks: int, max_splits: int = FD_MAX_SPLITS) -> int:
    return int(_load().fd_plan_splits(int(work_items), int(slots), int(n_kv_blocks), int(max_splits)))


def _host_i32(x):
    return np.ascontiguousarray(np.asarray(x, dtype=np.int32).reshape(-1))


def fd_plan(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, seqlens_host,
            num_sms: int = 0, *, block_table_host=None, page_size: int = 0) -> int:
    """Split count for one decode step (16-bit cache, one query per sequence).
    block_table_host: optional host [batch, max_pages_per_seq] int32 table of
    a paged cache with `page_size`-token pages; validated, never changes the plan."""
    sl = _host_i32(seqlens_host)
    if sl.shape[0] < batch:
        raise ValueError("seqlens_host shorter than batch")
    bt_ptr, mp = None, 0
    if block_table_host is not None:
        bt = np.ascontiguousarray(np.asarray(block_table_host, dtype=np.int32))
        if bt.ndim != 2 or bt.shape[0] < batch:
            raise ValueError("block_table_host must be [batch, max_pages_per_seq]")
        mp = bt.shape[1]
        bt_ptr = bt.ctypes.data
    r = _load().fd_plan(int(batch), int(n_q_heads), int(n_kv_heads), int(head_dim),
                        sl.ctypes.data if batch > 0 else None, bt_ptr, int(page_size), int(mp),
                        int(num_sms))
    return int(r)


def fd_plan_desc(desc: FdDesc, seqlens_host, num_sms: int = 0) -> int:
    """The split count fd_decode plans for `desc` (n_splits <= 0) with these lengths."""
    sl = _host_i32(seqlens_host)
    if sl.shape[0] < desc.batch:
        raise ValueError("seqlens_host shorter than batch")
    return int(_load().fd_plan_desc(ctypes.byref(desc), sl.ctypes.data if desc.batch > 0 else None,
                                    int(num_sms)))


def fd_workspace_size(desc: FdDesc, n_splits: int = 0) -> int:
    return int(_load().fd_workspace_size(ctypes.byref(desc), int(n_splits)))


def fd_decode(desc: FdDesc, q, k_cache, v_cache, seqlens, block_table, out, lse, workspace,
              workspace_bytes: int | None = None, stream=None) -> int:
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    return int(_load().fd_decode(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(seqlens), _ptr(block_table), _ptr(out), _ptr(lse),
                                 _ptr(workspace), int(wb), _stream(stream)))


def fd_split_states(desc: FdDesc, q, k_cache, v_cache, seqlens, block_table, workspace,
                    workspace_bytes: int | None = None, stream=None) -> int:
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    return int(_load().fd_split_states(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(seqlens), _ptr(block_table), _ptr(workspace),
                                       int(wb), _stream(stream)))


def fd_combine_states(desc: FdDesc, workspace, out, lse, workspace_bytes: int | None = None,
                      stream=None) -> int:
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    return int(_load().fd_combine_states(ctypes.byref(desc), _ptr(workspace), int(wb), _ptr(out),
                                         _ptr(lse), _stream(stream)))


def fd_decode_static(desc: FdDesc, q, k_cache, v_cache, seqlens, block_table, out, lse,
                     stream=None) -> int:
    """fd_decode without a caller workspace: for callers that cannot allocate
    device memory; the states go to the library's fixed device array
    (FD_STATIC_WORKSPACE_BYTES per GPU; not used at all with one split).
    Calls that overlap on the GPU race on that array."""
    return int(_load().fd_decode_static(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(seqlens), _ptr(block_table), _ptr(out), _ptr(lse),
                                        _stream(stream)))


def fd_decode_scaled(desc: FdDesc, scales: FdKvScales, q, k_cache, v_cache, seqlens, block_table, out, lse,
                     workspace, workspace_bytes: int | None = None, stream=None) -> int:
    """fd_decode over an E4M3 cache with a scale per (block of tokens, KV head); see make_scales."""
    _check_scales(desc, scales)
    _check_out(out, lse, desc.out_dtype, desc.batch * (desc.q_len or 1) * desc.n_q_heads)
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _load().fd_decode_scaled(ctypes.byref(desc), ctypes.byref(scales), _ptr(q), _ptr(k_cache),
                                    _ptr(v_cache), _ptr(seqlens), _ptr(block_table), _ptr(out), _ptr(lse),
                                    _ptr(workspace), wb, _stream(stream))


def fd_cache_store(desc: FdStoreDesc, scales: FdKvScales, k, v, slots, k_cache, v_cache, stream=None) -> int:
    """New K/V rows into an E4M3 cache at `slots` (int64), quantised with a power-of-two
    scale per (block of tokens, KV head); writes the cache and the scales."""
    _check_scales(desc, scales)
    if slots is not None and not isinstance(slots, int):
        if slots.element_size() != 8 or slots.numel() < desc.n_tokens or not slots.is_contiguous():
            raise ValueError(f"slots must be {desc.n_tokens} contiguous int64")
    return _load().fd_cache_store(ctypes.byref(desc), ctypes.byref(scales), _ptr(k), _ptr(v), _ptr(slots),
                                  _ptr(k_cache), _ptr(v_cache), _stream(stream))


def fd_page_tables(desc: FdPageDesc, seqlens, new_tokens, free_pages, free_count, block_table, seqlens_out,
                   free_count_out, cu_tokens, slots, positions, stream=None) -> int:
    """Pages for the new tokens of a step, and each new token's slot and position."""
    return int(_load().fd_page_tables(ctypes.byref(desc), _ptr(seqlens), _ptr(new_tokens), _ptr(free_pages),
                                      _ptr(free_count), _ptr(block_table), _ptr(seqlens_out),
                                      _ptr(free_count_out), _ptr(cu_tokens), _ptr(slots), _ptr(positions),
                                      _stream(stream)))


def fd_prompt_workspace_size(desc: FdPromptDesc) -> int:
    return int(_load().fd_prompt_workspace_size(ctypes.byref(desc)))


def fd_prompt(desc: FdPromptDesc, q, k, v, cu_q, cu_k, out, lse, workspace=None,
              workspace_bytes: int | None = None, stream=None) -> int:
    """Attention over whole prompts: packed sequences, causal or full."""
    _check_out(out, lse, desc.out_dtype, desc.total_q * desc.n_q_heads)
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _load().fd_prompt(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), _ptr(out),
                             _ptr(lse), _ptr(workspace), wb, _stream(stream))


def fd_device_status(stream=None, clear: bool = True) -> int:
    return int(_load().fd_device_status(_stream(stream), 1 if clear else 0))


def fd_decode_status(stream=None) -> int:
    return int(_load().fd_decode_status(_stream(stream)))


# ---------------------------------------------------------------- helpers
def _dtype_code(t) -> int:
    import torch
    codes = {torch.float16: FD_F16, torch.bfloat16: FD_BF16, torch.float32: FD_F32}
    if hasattr(torch, "float8_e4m3fn"):
        codes[torch.float8_e4m3fn] = FD_E4M3
    return codes[t]


def make_desc(q, k_cache, v_cache, *, n_kv_heads: int | None = None, page_size: int = 0,
              max_pages_per_seq: int = 0, max_seqlen: int = 0, n_splits: int = 0,
              out_dtype=None, k_scale: float = 1.0, v_scale: float = 1.0) -> FdDesc:
    """Descriptor for q [B, Hq, D] (or a query block [B, q_len, Hq, D]) and a
    cache given as 4-D strided tensors: contiguous [B, Hkv, T, D] (page_size 0)
    or a paged pool [P, Hkv, page, D] (any strided view of that shape, e.g. a
    permuted [P, page, Hkv, D]).  An fp8 cache (torch.float8_e4m3fn) takes
    k_scale / v_scale: key = k_scale * stored, value = v_scale * stored."""
    import torch
    d = FdDesc()
    if q.dim() == 4:
        B, q_len, Hq, D = q.shape
        d.q_len = q_len
        d.q_stride_t = q.stride(1)
        d.q_stride_b, d.q_stride_h = q.stride(0), q.stride(2)
    else:
        B, Hq, D = q.shape
        d.q_len = 1
        d.q_stride_t = 0
        d.q_stride_b, d.q_stride_h = q.stride(0), q.stride(1)
    d.batch, d.n_q_heads, d.head_dim = B, Hq, D
    d.n_kv_heads = int(n_kv_heads if n_kv_heads is not None else k_cache.shape[1])
    d.kv_dtype = _dtype_code(k_cache.dtype)
    d.out_dtype = _dtype_code(out_dtype if out_dtype is not None else torch.float32)
    d.k_stride_b, d.k_stride_h, d.k_stride_t = k_cache.stride(0), k_cache.stride(1), k_cache.stride(2)
    d.v_stride_b, d.v_stride_h, d.v_stride_t = v_cache.stride(0), v_cache.stride(1), v_cache.stride(2)
    if page_size:
        d.kv_extent = k_cache.shape[0]
        d.page_size = page_size
        d.max_pages_per_seq = max_pages_per_seq
    else:
        d.kv_extent = k_cache.shape[2]
        d.page_size = 0
        d.max_pages_per_seq = 0
    d.max_seqlen = int(max_seqlen)
    d.n_splits = int(n_splits)
    d.flags = 0
    d.q_dtype = _dtype_code(q.dtype)
    d.reserved = 0
    d.k_scale, d.v_scale = float(k_scale), float(v_scale)
    return d


def make_scales(k_scales, v_scales, *, block: int) -> FdKvScales:
    """Block scales of an E4M3 cache: float32 [P, Hkv, page / block] (paged) or
    [B, Hkv, ceil(T / block)] (contiguous), any strides.  The tensors are kept alive
    by the returned object."""
    import torch
    s = FdKvScales()
    for t in (k_scales, v_scales):
        if t.dim() != 3 or t.dtype != torch.float32:
            raise ValueError("scales must be float32 tensors of 3 dimensions")
    if k_scales.shape != v_scales.shape:
        raise ValueError("k_scales and v_scales must have the same shape")
    s.k, s.v = k_scales.data_ptr(), v_scales.data_ptr()
    s.k_stride_b, s.k_stride_h, s.k_stride_n = k_scales.stride()
    s.v_stride_b, s.v_stride_h, s.v_stride_n = v_scales.stride()
    s.block = int(block)
    s.reserved = 0
    s.shape = tuple(k_scales.shape)
    s._keep = (k_scales, v_scales)
    return s


def make_store_desc(k, v, k_cache, v_cache, *, page_size: int = 0) -> FdStoreDesc:
    """Descriptor for new rows k, v [n, Hkv, D] (16-bit, any strides with whole 16-byte
    rows) into an E4M3 cache [P, Hkv, page, D] (paged) or [B, Hkv, T, D] (page_size 0)."""
    d = FdStoreDesc()
    d.n_tokens, d.n_kv_heads, d.head_dim = k.shape
    if tuple(v.shape) != tuple(k.shape) or v.dtype != k.dtype:
        raise ValueError("k and v must have the same shape and type")
    for c in (k_cache, v_cache):
        if _dtype_code(c.dtype) != FD_E4M3 or c.dim() != 4 or c.shape[1] != d.n_kv_heads or c.shape[3] != d.head_dim:
            raise ValueError("the caches must be float8_e4m3fn tensors [pages or sequences, Hkv, tokens, D]")
        if page_size and c.shape[2] != page_size:
            raise ValueError("a paged cache's third dimension is its page size")
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must have the same shape")
    if k.stride(2) != 1 or v.stride(2) != 1 or k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("the head dimension must be contiguous")
    d.src_dtype = _dtype_code(k.dtype)
    d.k_src_stride_t, d.k_src_stride_h = k.stride(0), k.stride(1)
    d.v_src_stride_t, d.v_src_stride_h = v.stride(0), v.stride(1)
    d.k_stride_b, d.k_stride_h, d.k_stride_t = k_cache.stride()[:3]
    d.v_stride_b, d.v_stride_h, d.v_stride_t = v_cache.stride()[:3]
    d.page_size = int(page_size)
    d.kv_extent = k_cache.shape[0] if page_size else k_cache.shape[2]
    d.batch = k_cache.shape[0]
    return d


def make_page_desc(block_table, free_pages, slots, *, page_size: int, n_pages: int) -> FdPageDesc:
    """Descriptor for a table [B, max_pages_per_seq] (contiguous int32), the free stack (int32)
    and the slot map (int64)."""
    import torch
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous [B, max_pages_per_seq] tensor")
    if block_table.dtype != torch.int32 or free_pages.dtype != torch.int32 or not free_pages.is_contiguous():
        raise ValueError("block_table and free_pages must be contiguous int32 tensors")
    if slots.dtype != torch.int64 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int64 tensor")
    d = FdPageDesc()
    d.batch, d.max_pages_per_seq = block_table.shape
    d.page_size, d.n_pages = int(page_size), int(n_pages)
    d.n_free_max, d.n_slots = free_pages.numel(), slots.numel()
    return d


def make_prompt_desc(q, k, v, *, batch: int, causal: bool = True, max_q: int = 0, max_k: int = 0,
                     n_splits: int = 0, out_dtype=None) -> FdPromptDesc:
    """Descriptor for packed prompts q [total_q, Hq, D], k and v [total_k, Hkv, D]
    (16-bit; any strides with a contiguous head dimension, so slices of one
    projection's output too, but no expanded heads: those are one KV head)."""
    import torch
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k and v must have one type")
    if k.shape != v.shape or q.shape[2] != k.shape[2]:
        raise ValueError("q [total_q, Hq, D], k and v [total_k, Hkv, D]")
    if q.stride(2) != 1 or k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("the head dimension must be contiguous")
    d = FdPromptDesc()
    d.batch = int(batch)
    d.total_q, d.n_q_heads, d.head_dim = q.shape
    d.total_k, d.n_kv_heads = k.shape[:2]
    d.dtype = _dtype_code(q.dtype)
    d.out_dtype = _dtype_code(out_dtype if out_dtype is not None else torch.float32)
    d.q_stride_t, d.q_stride_h = q.stride(0), q.stride(1)
    d.k_stride_t, d.k_stride_h = k.stride(0), k.stride(1)
    d.v_stride_t, d.v_stride_h = v.stride(0), v.stride(1)
    d.max_q, d.max_k = int(max_q), int(max_k)
    d.causal, d.n_splits = int(bool(causal)), int(n_splits)
    d.flags = d.reserved = 0
    return d
