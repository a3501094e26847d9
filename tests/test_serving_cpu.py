"""The serving entry points on the host: struct layouts, and every refusal
before anything is enqueued.  CPU only (a refused call makes no CUDA call)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def fd():
    import split_kv_gb300
    from split_kv_gb300 import _build
    _build.build()
    return split_kv_gb300


def test_struct_sizes_match_the_header(fd):
    assert ctypes.sizeof(fd.FdKvScales) == 72        # 2 pointers, 6 int64, 2 int32
    assert ctypes.sizeof(fd.FdStoreDesc) == 112      # 4 int32, 11 int64, 2 int32
    assert ctypes.sizeof(fd.FdPageDesc) == 24
    assert ctypes.sizeof(fd.FdPromptDesc) == 104     # 6 int32, 6 int64, 8 int32


def _prompt(fd):
    d = fd.FdPromptDesc()
    d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim = 1, 8, 2, 128
    d.dtype, d.out_dtype = fd.FD_BF16, fd.FD_F32
    d.q_stride_t, d.q_stride_h = 1024, 128
    d.k_stride_t, d.k_stride_h = 256, 128
    d.v_stride_t, d.v_stride_h = 256, 128
    d.total_q = d.total_k = 64
    d.causal = 1
    return d


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, -1), ("n_kv_heads", 3, -1), ("n_q_heads", 0, -1), ("head_dim", 64, -2), ("dtype", 2, -2),
    ("dtype", 9, -1), ("out_dtype", 3, -1), ("q_stride_t", 100, -1), ("k_stride_h", 4, -1), ("v_stride_t", 64, -1),
    ("total_q", -1, -1), ("causal", 2, -1), ("flags", 1, -1), ("reserved", 1, -1), ("n_splits", 129, -2),
    ("n_splits", 2, -3)])
def test_prompt_refuses(fd, field, value, status):
    d = _prompt(fd)
    setattr(d, field, value)
    assert fd.fd_prompt(d, 1024, 1024, 1024, 1024, 1024, 1024, None, None, 0, stream=0) == status


def test_prompt_refuses_pointers_and_sizes_its_workspace(fd):
    d = _prompt(fd)
    for bad in range(6):
        a = [1024] * 6
        a[bad] = None
        assert fd.fd_prompt(d, *a, None, None, 0, stream=0) == fd.FD_ERR_INVALID_ARG
    assert fd.fd_prompt(d, 1032, 1024, 1024, 1024, 1024, 1024, None, None, 0, stream=0) == fd.FD_ERR_INVALID_ARG
    assert fd.fd_prompt_workspace_size(d) == 0
    d.n_splits = 3
    assert fd.fd_prompt_workspace_size(d) == 64 * 8 * 3 * 130 * 4
    d.batch = 0
    assert fd.fd_prompt(d, 1024, 1024, 1024, 1024, 1024, 1024, None, None, 0, stream=0) == fd.FD_OK


def _scales(fd, block=16):
    s = fd.FdKvScales()
    s.k = s.v = 1024
    s.k_stride_b = s.v_stride_b = 8
    s.k_stride_h = s.v_stride_h = 4
    s.k_stride_n = s.v_stride_n = 1
    s.block = block
    return s


def _store(fd):
    d = fd.FdStoreDesc()
    d.n_tokens, d.n_kv_heads, d.head_dim, d.src_dtype = 4, 2, 128, fd.FD_F16
    d.k_src_stride_t = d.v_src_stride_t = 256
    d.k_src_stride_h = d.v_src_stride_h = 128
    d.k_stride_b = d.v_stride_b = 16384
    d.k_stride_h = d.v_stride_h = 8192
    d.k_stride_t = d.v_stride_t = 128
    d.kv_extent, d.page_size = 10, 64
    return d


@pytest.mark.parametrize("field,value,status", [
    ("n_tokens", -1, -1), ("n_kv_heads", 0, -1), ("head_dim", 64, -2), ("src_dtype", 2, -2), ("src_dtype", 7, -1),
    ("page_size", 12, -1), ("page_size", 4, -2), ("kv_extent", 0, -1), ("k_src_stride_t", 3, -1),
    ("v_stride_h", 8, -1), ("k_stride_t", 64, -1), ("page_size", 0, -1), ("n_tokens", 0, 0)])
def test_store_refuses(fd, field, value, status):
    d = _store(fd)
    setattr(d, field, value)
    assert fd.fd_cache_store(d, _scales(fd), 1024, 1024, 1024, 1024, 1024, stream=0) == status


@pytest.mark.parametrize("field,value,status", [
    ("k", None, -1), ("v", 1026, -1), ("block", 0, -1), ("block", 24, -1), ("block", 128, -1), ("block", 2048, -2),
    ("k_stride_n", -1, -1), ("reserved", 1, -1)])
def test_scales_are_checked_by_the_store_and_the_decode(fd, field, value, status):
    s = _scales(fd)
    setattr(s, field, value)
    assert fd.fd_cache_store(_store(fd), s, 1024, 1024, 1024, 1024, 1024, stream=0) == status
    d = fd.FdDesc()
    d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim, d.kv_dtype, d.q_dtype = 1, 8, 2, 128, fd.FD_E4M3, fd.FD_F16
    d.q_stride_b, d.q_stride_h = 1024, 128
    d.k_stride_b = d.v_stride_b = 16384
    d.k_stride_h = d.v_stride_h = 8192
    d.k_stride_t = d.v_stride_t = 128
    d.kv_extent, d.page_size, d.max_pages_per_seq, d.n_splits, d.k_scale, d.v_scale = 10, 64, 4, 1, 1.0, 1.0
    assert fd.fd_decode_scaled(d, s, 1024, 1024, 1024, 1024, 1024, 1024, None, None, 0, stream=0) == status
    d.kv_dtype = fd.FD_F16
    assert fd.fd_decode_scaled(d, _scales(fd), 1024, 1024, 1024, 1024, 1024, 1024, None, None, 0,
                               stream=0) == fd.FD_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, -1), ("batch", 8193, -2), ("page_size", 12, -1), ("page_size", 4, -2), ("max_pages_per_seq", 0, -1),
    ("max_pages_per_seq", 1 << 28, -1), ("n_pages", 0, -1), ("n_free_max", -1, -1), ("n_slots", -1, -1)])
def test_tables_refuse(fd, field, value, status):
    d = fd.FdPageDesc()
    d.batch, d.page_size, d.max_pages_per_seq, d.n_pages, d.n_free_max, d.n_slots = 2, 16, 8, 20, 4, 10
    setattr(d, field, value)
    assert fd.fd_page_tables(d, *[1024] * 10, stream=0) == status
    for bad in range(9):
        if bad == 7:
            continue                                   # cu_tokens may be absent
        d2 = fd.FdPageDesc()
        d2.batch, d2.page_size, d2.max_pages_per_seq, d2.n_pages, d2.n_free_max, d2.n_slots = 2, 16, 8, 20, 4, 10
        a = [1024] * 10
        a[bad] = None
        assert fd.fd_page_tables(d2, *a, stream=0) == fd.FD_ERR_INVALID_ARG
