"""split_kv_gb300 -- split-KV decode attention (Flash-Decoding) for GB300.

A thin ctypes binding over the C ABI of ``lib/libfd.so`` (declared in
``include/fd.h``).  Every function has the C name and does argument
marshalling only: torch tensors are passed as device pointers, streams as
``cudaStream_t`` handles, and every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback: if the library is missing
the first call raises.

A paged cache's life around the decode: fd_page_tables gives pages to new tokens, fd_qkv_rope and
fd_cache_store fill them, fd_page_fork shares them, fd_page_trim gives them back, fd_page_compact and
fd_page_copy move them.

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
FD_NORM_Q, FD_NORM_K = 1, 2
FD_MAX_TABLE_BATCH = 8192
FD_MAX_COMPACT_PAGES = 1 << 19

LIB_PATH = _build.LIB_PATH

# every function the header declares (checked against include/fd.h by the tests)
EXPORTS = ("fd_abi_version", "fd_status_string", "fd_num_sms", "fd_plan_splits", "fd_plan",
           "fd_plan_desc", "fd_workspace_size", "fd_decode", "fd_split_states", "fd_combine_states",
           "fd_device_status", "fd_decode_status", "fd_decode_static", "fd_decode_scaled",
           "fd_cache_store", "fd_page_tables", "fd_prompt", "fd_prompt_workspace_size", "fd_qkv_rope",
           "fd_page_fork", "fd_page_trim", "fd_page_compact", "fd_page_copy")


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
    copy_list = False       # make_page_desc: n_slots counts a copy list, not a slot map


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


class FdRopeDesc(ctypes.Structure):
    """Mirror of ``fd_rope_desc`` (include/fd.h)."""
    _fields_ = [
        *((n, ctypes.c_int32) for n in ("n_tokens", "n_q_heads", "n_kv_heads", "head_dim", "dtype", "cache_dtype",
                                        "w_dtype", "norm", "rot_dim", "interleaved")),
        *((n, ctypes.c_float) for n in ("eps", "rot_scale", "k_scale", "v_scale")),
        *((n, ctypes.c_int64) for n in (
            "q_stride_t", "q_stride_h", "k_src_stride_t", "k_src_stride_h", "v_src_stride_t", "v_src_stride_h",
            "q_out_stride_t", "q_out_stride_h", "k_out_stride_t", "k_out_stride_h",
            "k_stride_b", "k_stride_h", "k_stride_t", "v_stride_b", "v_stride_h", "v_stride_t",
            "q_w_stride_h", "k_w_stride_h", "kv_extent")),
        *((n, ctypes.c_int32) for n in ("page_size", "batch", "flags", "reserved")),
    ]
    sizes = None            # make_rope_desc: bytes of a token's queries and of its keys, of a cache; the weights' type, and
                            # how many there are for queries and keys (0: not used)


class FdPool(ctypes.Structure):
    """Mirror of ``fd_pool`` (include/fd.h)."""
    _fields_ = [("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("stride", ctypes.c_int64 * 2),
                ("extent", ctypes.c_int32 * 2), ("row_bytes", ctypes.c_int32), ("reserved", ctypes.c_int32)]


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
            "fd_qkv_rope": (i32, [ctypes.POINTER(FdRopeDesc)] + [vp] * 13),
            "fd_page_fork": (i32, [ctypes.POINTER(FdPageDesc), i32] + [vp] * 14),
            "fd_page_trim": (i32, [ctypes.POINTER(FdPageDesc)] + [vp] * 12),
            "fd_page_compact": (i32, [ctypes.POINTER(FdPageDesc), i32] + [vp] * 10),
            "fd_page_copy": (i32, [ctypes.POINTER(FdPool), i32, i32, i32, vp, vp, vp, vp]),
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


_types = {}
_int32 = _int64 = _float32 = None


def _array(t, n: int, name: str, kind: str):
    """Address of n contiguous elements of the type, checked if t is a tensor (addresses and None go
    unchecked)."""
    global _int32, _int64, _float32
    if t is None:
        return None
    try:
        dtype = t.dtype
    except AttributeError:
        return _ptr(t)
    if not _types:
        import torch
        _types.update(int32=torch.int32, int64=torch.int64, float32=torch.float32)
        _int32, _int64, _float32 = torch.int32, torch.int64, torch.float32
    if dtype is not _types[kind] or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous {kind}")
    return t.data_ptr()


def _flat(t, n: int, name: str, dtype, kind: str):
    """_array, the short way (dtype: what kind names, None before the first call)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.numel() >= n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _array(t, n, name, kind)


def _i32(t, n: int, name: str):
    """_flat of int32."""
    if t is None:
        return None
    try:
        if t.dtype is _int32 and t.numel() >= n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _array(t, n, name, "int32")


def _room(t, size: int, name: str):
    """Address of a strided tensor that holds `size` bytes or more (addresses and None go unchecked)."""
    if t is None:
        return None
    try:
        if t.nbytes >= size:
            return t.data_ptr()
    except AttributeError:
        return _ptr(t)
    raise ValueError(f"{name} must hold {size} bytes, as its descriptor says")


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
    if desc.copy_list:
        raise ValueError("fd_page_tables takes a descriptor of a slot map, this one is of a copy list")
    b, n = desc.batch, desc.n_slots
    return _load().fd_page_tables(ctypes.byref(desc), _i32(seqlens, b, "seqlens"), _i32(new_tokens, b, "new_tokens"),
                                  _i32(free_pages, desc.n_free_max, "free_pages"), _i32(free_count, 1, "free_count"),
                                  _i32(block_table, b * desc.max_pages_per_seq, "block_table"), _i32(seqlens_out, b, "seqlens_out"),
                                  _i32(free_count_out, 1, "free_count_out"), _i32(cu_tokens, b + 1, "cu_tokens"),
                                  _flat(slots, n, "slots", _int64, "int64"), _i32(positions, n, "positions"), _stream(stream))


def fd_prompt_workspace_size(desc: FdPromptDesc) -> int:
    return int(_load().fd_prompt_workspace_size(ctypes.byref(desc)))


def fd_prompt(desc: FdPromptDesc, q, k, v, cu_q, cu_k, out, lse, workspace=None,
              workspace_bytes: int | None = None, stream=None) -> int:
    """Attention over whole prompts: packed sequences, causal or full."""
    _check_out(out, lse, desc.out_dtype, desc.total_q * desc.n_q_heads)
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _load().fd_prompt(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), _ptr(out),
                             _ptr(lse), _ptr(workspace), wb, _stream(stream))


def fd_qkv_rope(desc: FdRopeDesc, q, k, v, q_weight, k_weight, inv_freq, positions, slots, q_out, k_out, k_cache,
                v_cache, stream=None) -> int:
    """Norms and rotation of a step's queries and keys, and the way of its keys and values into a cache."""
    n = desc.n_tokens
    if desc.sizes is None:              # a descriptor of the caller's own: as for addresses
        q_row = k_row = cache = 0
    else:
        q_row, k_row, cache, kind, q_weights, k_weights = desc.sizes
        q_row, k_row = n * q_row, n * k_row
        try:
            if ((q_weight is not None and q_weights and (q_weight.dtype is not kind or q_weight.numel() < q_weights)) or
                    (k_weight is not None and k_weights and (k_weight.dtype is not kind or k_weight.numel() < k_weights))):
                raise ValueError("q_weight and k_weight must have the type and size of their descriptor's weights")
        except AttributeError:
            pass
    return _load().fd_qkv_rope(ctypes.byref(desc), _room(q, q_row, "q"), _room(k, k_row, "k"), _room(v, k_row if cache else 0, "v"),
                               _ptr(q_weight), _ptr(k_weight), _flat(inv_freq, desc.rot_dim // 2, "inv_freq", _float32, "float32"),
                               _i32(positions, n, "positions"), _flat(slots, n, "slots", _int64, "int64"), _room(q_out, q_row, "q_out"),
                               _room(k_out, k_row, "k_out"), _room(k_cache, cache, "k_cache"), _room(v_cache, cache, "v_cache"),
                               _stream(stream))


def _page_arrays(desc, free_pages, free_count, block_table, shares, free_count_out, copy_src, copy_dst, copy_count):
    """Addresses of what fd_page_fork, _trim and _compact take alike, as large as their descriptor says."""
    n = desc.n_slots
    return (_i32(free_pages, desc.n_free_max, "free_pages"), _i32(free_count, 1, "free_count"),
            _i32(block_table, desc.batch * desc.max_pages_per_seq, "block_table"), _i32(shares, desc.n_pages, "shares"),
            _i32(free_count_out, 1, "free_count_out"), _i32(copy_src, n, "copy_src"), _i32(copy_dst, n, "copy_dst"),
            _i32(copy_count, 1, "copy_count"))


def fd_page_fork(desc: FdPageDesc, parents, children, keep, seqlens, free_pages, free_count, block_table, shares, seqlens_out,
                 free_count_out, copy_src, copy_dst, copy_count, n_forks: int | None = None, stream=None) -> int:
    """Sequences children[i] that share the pages of parents[i]'s first keep[i] tokens (None: of all)."""
    n = parents.numel() if n_forks is None else int(n_forks)
    b = desc.batch
    free, count, table, held, count_out, src, dst, copies = _page_arrays(desc, free_pages, free_count, block_table, shares, free_count_out,
                                                                         copy_src, copy_dst, copy_count)
    return _load().fd_page_fork(ctypes.byref(desc), n, _i32(parents, n, "parents"), _i32(children, n, "children"), _i32(keep, n, "keep"),
                                _i32(seqlens, b, "seqlens"), free, count, table, held, _i32(seqlens_out, b, "seqlens_out"), count_out, src,
                                dst, copies, _stream(stream))


def fd_page_trim(desc: FdPageDesc, keep, seqlens, free_pages, free_count, block_table, shares, seqlens_out, free_count_out,
                 copy_src=None, copy_dst=None, copy_count=None, stream=None) -> int:
    """Sequences cut to their first keep[b] tokens; pages that nobody holds any more go back to the free stack."""
    b = desc.batch
    free, count, table, held, count_out, src, dst, copies = _page_arrays(desc, free_pages, free_count, block_table, shares, free_count_out,
                                                                         copy_src, copy_dst, copy_count)
    return _load().fd_page_trim(ctypes.byref(desc), _i32(keep, b, "keep"), _i32(seqlens, b, "seqlens"), free, count, table, held,
                                _i32(seqlens_out, b, "seqlens_out"), count_out, src, dst, copies, _stream(stream))


def fd_page_compact(desc: FdPageDesc, n_keep: int, seqlens, free_pages, free_count, block_table, shares, free_count_out,
                    copy_src, copy_dst, copy_count, stream=None) -> int:
    """Held pages from n_keep on renamed to free pages below it, for the high end of a pool to be given up."""
    return _load().fd_page_compact(ctypes.byref(desc), int(n_keep), _i32(seqlens, desc.batch, "seqlens"),
                                   *_page_arrays(desc, free_pages, free_count, block_table, shares, free_count_out, copy_src, copy_dst,
                                                 copy_count), _stream(stream))


def fd_page_copy(pools, copy_src, copy_dst, copy_count=None, n_pairs: int | None = None, stream=None) -> int:
    """Page copy_dst[i] of every pool (make_pools) becomes what page copy_src[i] is."""
    n = copy_src.numel() if n_pairs is None else int(n_pairs)
    return _load().fd_page_copy(pools, len(pools), pools.n_pages, n, _i32(copy_src, n, "copy_src"), _i32(copy_dst, n, "copy_dst"),
                                _i32(copy_count, 1, "copy_count"), _stream(stream))


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


def make_page_desc(block_table, free_pages, slots, *, page_size: int, n_pages: int, copies=None) -> FdPageDesc:
    """Descriptor for a table [B, max_pages_per_seq] (contiguous int32), the free stack (int32)
    and the slot map (int64) of fd_page_tables, or, with slots None, the copy list's
    arrays (copies: one of them, int32; None: no list) of fd_page_fork, _trim and _compact."""
    import torch
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous [B, max_pages_per_seq] tensor")
    if block_table.dtype != torch.int32 or free_pages.dtype != torch.int32 or not free_pages.is_contiguous():
        raise ValueError("block_table and free_pages must be contiguous int32 tensors")
    if slots is not None:
        if slots.dtype != torch.int64 or not slots.is_contiguous():
            raise ValueError("slots must be a contiguous int64 tensor")
        if copies is not None:
            raise ValueError("a descriptor has a slot map or a copy list")
    elif copies is not None and (copies.dtype != torch.int32 or not copies.is_contiguous()):
        raise ValueError("copies must be a contiguous int32 tensor")
    d = FdPageDesc()
    d.batch, d.max_pages_per_seq = block_table.shape
    d.page_size, d.n_pages = int(page_size), int(n_pages)
    d.n_free_max = free_pages.numel()
    d.n_slots = slots.numel() if slots is not None else copies.numel() if copies is not None else 0
    d.copy_list = slots is None
    return d


def make_rope_desc(q, k, v=None, *, q_out=None, k_out=None, k_cache=None, v_cache=None, page_size: int = 0, q_weight=None,
                   k_weight=None, norm_q: bool = True, norm_k: bool = True, rot_dim: int = 128, interleaved: bool = False,
                   eps: float = 1e-6, rot_scale: float = 1.0, k_scale: float = 1.0, v_scale: float = 1.0) -> FdRopeDesc:
    """Descriptor for a step's heads q [n, Hq, D], k and v [n, Hkv, D] (16-bit, any strides with
    whole 16-byte rows; q or k may be None), rows out q_out and k_out of their shapes, caches
    [P, Hkv, page, D] (paged) or [B, Hkv, T, D] (page_size 0) of their type or float8_e4m3fn,
    and weights [D] or [heads, D]."""
    import torch
    d = FdRopeDesc()
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    d.n_tokens, _, d.head_dim = x.shape
    d.dtype = _dtype_code(x.dtype)
    if (k_cache is None) != (v_cache is None) or (k_cache is not None and (v is None or k is None)):
        raise ValueError("a cache takes k, v, k_cache and v_cache")
    if q is not None and q_out is None or k is not None and k_out is None and k_cache is None:
        raise ValueError("q needs q_out, k needs k_out or caches")
    for name, t, like in (("q", q, None), ("k", k, None), ("v", v if k_cache is not None else None, k), ("q_out", q_out, q),
                          ("k_out", k_out, k)):
        if t is None:
            continue
        if t.dim() != 3 or t.shape[0] != d.n_tokens or t.shape[2] != d.head_dim or t.dtype != x.dtype or t.stride(2) != 1:
            raise ValueError(f"{name} must be [{d.n_tokens}, heads, {d.head_dim}] of one 16-bit type, the head dimension contiguous")
        if name not in "qk" and (like is None or t.shape != like.shape):
            raise ValueError(f"{name} must have the shape of its rows")
    d.n_q_heads = 0 if q is None else q.shape[1]
    d.n_kv_heads = 0 if k is None else k.shape[1]
    if q is not None:
        d.q_stride_t, d.q_stride_h = q.stride()[:2]
        d.q_out_stride_t, d.q_out_stride_h = q_out.stride()[:2]
    if k is not None:
        d.k_src_stride_t, d.k_src_stride_h = k.stride()[:2]
        if k_out is not None:
            d.k_out_stride_t, d.k_out_stride_h = k_out.stride()[:2]
    d.cache_dtype = d.dtype
    if k_cache is not None:
        d.v_src_stride_t, d.v_src_stride_h = v.stride()[:2]
        if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
            raise ValueError("k_cache and v_cache must have the same shape and type")
        if k_cache.dim() != 4 or k_cache.shape[1] != d.n_kv_heads or k_cache.shape[3] != d.head_dim:
            raise ValueError("the caches must be [pages or sequences, Hkv, tokens, D]")
        if k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
            raise ValueError("the head dimension must be contiguous")
        if page_size and k_cache.shape[2] != page_size:
            raise ValueError("a paged cache's third dimension is its page size")
        d.cache_dtype = _dtype_code(k_cache.dtype)
        d.k_stride_b, d.k_stride_h, d.k_stride_t = k_cache.stride()[:3]
        d.v_stride_b, d.v_stride_h, d.v_stride_t = v_cache.stride()[:3]
        d.page_size = int(page_size)
        d.kv_extent = k_cache.shape[0] if page_size else k_cache.shape[2]
        d.batch = k_cache.shape[0]
    d.norm = (FD_NORM_Q if norm_q and q is not None else 0) | (FD_NORM_K if norm_k and k is not None else 0)
    d.w_dtype = FD_F32
    types = set()
    for name, w, heads in (("q_weight", q_weight, d.n_q_heads), ("k_weight", k_weight, d.n_kv_heads)):
        if w is None:
            continue
        if w.shape[-1] != d.head_dim or w.dim() > 2 or w.stride(-1) != 1 or (w.dim() == 2 and w.shape[0] != heads):
            raise ValueError(f"{name} must be [D] or [heads, D], the last dimension contiguous")
        types.add(w.dtype)
        if w.dim() == 2 and heads > 1:
            setattr(d, name[0] + "_w_stride_h", w.stride(0))
        d.w_dtype = _dtype_code(w.dtype)
    if len(types) > 1:
        raise ValueError("q_weight and k_weight must have one type")
    count = lambda used, heads, stride: 0 if not used else d.head_dim * (heads if stride else 1)
    d.sizes = (2 * d.head_dim * d.n_q_heads, 2 * d.head_dim * d.n_kv_heads, 0 if k_cache is None else k_cache.nbytes,
               types.pop() if types else torch.float32, count(d.norm & FD_NORM_Q, d.n_q_heads, d.q_w_stride_h),
               count(d.norm & FD_NORM_K, d.n_kv_heads, d.k_w_stride_h))
    d.rot_dim, d.interleaved = int(rot_dim), int(bool(interleaved))
    d.eps, d.rot_scale, d.k_scale, d.v_scale = float(eps), float(rot_scale), float(k_scale), float(v_scale)
    d.flags = d.reserved = 0
    return d


def make_pools(tensors):
    """Pools of fd_page_copy: tensors [P, ...] of up to four dimensions with one number of pages
    (a layer's K or V cache [P, Hkv, page, D] in any order of storage, its scales [P, Hkv,
    page / block]).  The tensors are kept alive by the returned array."""
    tensors = list(tensors)
    pools = (FdPool * len(tensors))()
    pages = {t.shape[0] for t in tensors}
    if len(pages) > 1 or 0 in pages:
        raise ValueError("the pools must have one number of pages")
    for x, t in zip(pools, tensors):
        size = t.element_size()
        inner = [(n, st * size) for n, st in zip(t.shape[1:], t.stride()[1:]) if n != 1]
        if 0 in t.shape or len(inner) > 3:
            raise ValueError("a pool is a tensor [pages, ...] of up to four dimensions, none of them empty")
        x.row_bytes = size
        if inner and inner[-1][1] == size:
            x.row_bytes *= inner.pop()[0]
        if len(inner) > 2:
            raise ValueError("a pool's last dimension must be contiguous")
        inner = [(1, 0)] * (2 - len(inner)) + inner
        x.base = t.data_ptr()
        x.page_stride = t.stride(0) * size if t.shape[0] > 1 else max(1, t.stride(0)) * size
        for i, (n, st) in enumerate(inner):
            x.extent[i], x.stride[i] = n, st
        x.reserved = 0
    pools.n_pages = pages.pop() if pages else 1
    pools._keep = tensors
    return pools


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
