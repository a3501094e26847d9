"""Layouts that the kernels cannot address, refused on the host.  CPU only."""
import pytest
import torch

from test_serving_cpu import _prompt, _scales, _store, fd  # noqa: F401


def _decode(fd, **kw):
    d = fd.FdDesc()
    d.batch, d.n_q_heads, d.n_kv_heads, d.head_dim = 3, 32, 8, 128
    d.kv_dtype = d.q_dtype = fd.FD_F16
    d.q_stride_b, d.q_stride_h = 32 * 128, 128
    d.k_stride_b = d.v_stride_b = 8 * 64 * 128
    d.k_stride_h = d.v_stride_h = 64 * 128
    d.k_stride_t = d.v_stride_t = 128
    d.kv_extent, d.n_splits, d.k_scale, d.v_scale = 64, 2, 1.0, 1.0
    for name, value in kw.items():
        setattr(d, name, value)
    return d


@pytest.mark.parametrize("field", ["q_stride_h", "k_stride_h", "v_stride_h"])
def test_prompt_refuses_heads_that_share_their_rows(fd, field):  # noqa: F811
    """A head stride of 0 (torch's expand) has no tensor map; with one head it is never used."""
    d = _prompt(fd)
    setattr(d, field, 0)
    assert fd.fd_prompt(d, 1024, 1024, 1024, 1024, 1024, 1024, None, None, 0, stream=0) == fd.FD_ERR_INVALID_ARG
    assert fd.fd_prompt_workspace_size(d) == 0
    d = _prompt(fd)
    d.n_q_heads = d.n_kv_heads = 1
    d.n_splits = 3
    setattr(d, field, 0)
    assert fd.fd_prompt_workspace_size(d) > 0


def test_prompt_refuses_an_expanded_tensor(fd):  # noqa: F811
    q, k = torch.zeros(4, 8, 128, dtype=torch.float16), torch.zeros(4, 1, 128, dtype=torch.float16)
    d = fd.make_prompt_desc(q, k.expand(-1, 8, -1), k.expand(-1, 8, -1), batch=1)
    assert fd.fd_prompt(d, 1024, 1024, 1024, 1024, 1024, 1024, None, None, 0, stream=0) == fd.FD_ERR_INVALID_ARG


@pytest.mark.parametrize("field", ["k_stride_b", "k_stride_h", "v_stride_b", "v_stride_h"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_refuses_a_cache_that_shares_its_rows(fd, field, paged, fp8):  # noqa: F811
    kw = {field: 0}
    if paged:
        kw.update(page_size=64, max_pages_per_seq=4, kv_extent=9)
    if fp8:
        kw.update(kv_dtype=fd.FD_E4M3)
    d = _decode(fd, **kw)
    table = 1024 if paged else None
    args = (1024, 1024, 1024, 1024, table, 1024, 1024, 1024, 1 << 30)
    assert fd.fd_decode(d, *args, stream=0) == fd.FD_ERR_INVALID_ARG
    assert fd.fd_split_states(d, 1024, 1024, 1024, 1024, table, 1024, 1 << 30, stream=0) == fd.FD_ERR_INVALID_ARG
    if fp8:
        assert fd.fd_decode_scaled(d, _scales(fd), *args, stream=0) == fd.FD_ERR_INVALID_ARG


def test_store_of_no_rows_takes_empty_tensors(fd):  # noqa: F811
    """A step without new rows: the address of an empty tensor is null."""
    d = _store(fd)
    d.n_tokens = 0
    for k, v, slots, kc, vc in ((None, None, None, 1024, 1024), (1024, 1024, None, 1024, 1024), (None,) * 5):
        assert fd.fd_cache_store(d, _scales(fd), k, v, slots, kc, vc, stream=0) == fd.FD_OK
    d.n_tokens = 1
    assert fd.fd_cache_store(d, _scales(fd), 1024, 1024, None, 1024, 1024, stream=0) == fd.FD_ERR_INVALID_ARG
    none = torch.empty(0, 2, 128, dtype=torch.float16)
    kc, vc = (torch.zeros(10, 2, 64, 128).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = torch.ones(10, 2, 4), torch.ones(10, 2, 4)
    d = fd.make_store_desc(none, none, kc, vc, page_size=64)
    slots = torch.empty(0, dtype=torch.int64)
    assert fd.fd_cache_store(d, fd.make_scales(ks, vs, block=16), none, none, slots, kc, vc, stream=0) == fd.FD_OK


def test_scaled_decode_of_no_sequences_takes_empty_tensors(fd):  # noqa: F811
    d = _decode(fd, batch=0, kv_dtype=fd.FD_E4M3, page_size=64, max_pages_per_seq=4)
    assert fd.fd_decode_scaled(d, _scales(fd), None, 1024, 1024, None, None, None, None, None, 0, stream=0) == fd.FD_OK
    d.batch = 1
    assert fd.fd_decode_scaled(d, _scales(fd), None, 1024, 1024, 1024, 1024, 1024, None, 1024, 1 << 30,
                               stream=0) == fd.FD_ERR_INVALID_ARG


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("field", ["k_stride_b", "k_stride_h", "v_stride_b", "v_stride_h"])
def test_store_refuses_a_cache_that_shares_its_rows(fd, field, paged):  # noqa: F811
    """Rows of two pages or heads in one place: which of them it keeps would be chance."""
    d = _store(fd)
    if not paged:
        d.page_size, d.kv_extent, d.batch = 0, 64, 5
    setattr(d, field, 0)
    assert fd.fd_cache_store(d, _scales(fd), 1024, 1024, 1024, 1024, 1024, stream=0) == fd.FD_ERR_INVALID_ARG


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("field", ["k_stride_b", "k_stride_h", "k_stride_n", "v_stride_b", "v_stride_h", "v_stride_n"])
def test_store_refuses_scales_that_several_blocks_share(fd, field, paged):  # noqa: F811
    """The decode may read one scale for many blocks, the store writes each block's own."""
    d, s = _store(fd), _scales(fd)
    if not paged:
        d.page_size, d.kv_extent, d.batch = 0, 64, 5
    setattr(s, field, 0)
    assert fd.fd_cache_store(d, s, 1024, 1024, 1024, 1024, 1024, stream=0) == fd.FD_ERR_INVALID_ARG


# ------------------------------------------------------------------ the binding's own checks
def test_page_desc_refuses_other_types(fd):  # noqa: F811
    """The kernel writes 8 bytes a slot and reads 4 a page: tensors of other types are shorter or longer than they look."""
    i32, i64 = (lambda *n: torch.zeros(*n, dtype=torch.int32)), (lambda *n: torch.zeros(*n, dtype=torch.int64))
    d = fd.make_page_desc(i32(2, 8), i32(4), i64(10), page_size=16, n_pages=20)
    assert (d.batch, d.max_pages_per_seq, d.n_free_max, d.n_slots) == (2, 8, 4, 10)
    for table, free, slots in ((i32(2, 8), i32(4), i32(10)), (i64(2, 8), i32(4), i64(10)), (i32(2, 8), i64(4), i64(10)),
                               (i32(2, 8), i32(4), i64(20)[::2]), (i32(2, 8), i32(8)[::2], i64(10)), (i32(16), i32(4), i64(10))):
        with pytest.raises(ValueError):
            fd.make_page_desc(table, free, slots, page_size=16, n_pages=20)


@pytest.mark.parametrize("page", [64, 0])
def test_scales_and_slots_have_to_cover_the_call(fd, page):  # noqa: F811
    """The C ABI sees addresses only; the binding has the tensors and compares them."""
    kc, vc = (torch.zeros(3, 2, 64, 128).to(torch.float8_e4m3fn) for _ in range(2))
    rows = torch.zeros(5, 2, 128, dtype=torch.float16)
    store = fd.make_store_desc(rows, rows, kc, vc, page_size=page)
    q = torch.zeros(3, 8, 128, dtype=torch.float16)
    decode = fd.make_desc(q, kc, vc, page_size=page, max_pages_per_seq=2, max_seqlen=64, n_splits=1)
    store_0, decode_0 = fd.FdStoreDesc.from_buffer_copy(store), decode.copy()
    store_0.n_tokens, decode_0.batch = 0, 0                    # (nothing is enqueued: the checks alone)
    scales = lambda *n: fd.make_scales(torch.ones(*n), torch.ones(*n), block=16)
    slots = torch.zeros(5, dtype=torch.int64)
    call_store = lambda d, s, at: fd.fd_cache_store(d, s, rows, rows, at, kc, vc, stream=0)
    call_decode = lambda d, s: fd.fd_decode_scaled(d, s, q, kc, vc, 1024, 1024, 1024, None, None, 0, stream=0)
    assert call_store(store_0, scales(3, 2, 4), slots) == fd.FD_OK
    assert call_decode(decode_0, scales(3, 2, 4)) == fd.FD_OK
    for n in ((2, 2, 4), (3, 1, 4), (3, 2, 3)):
        with pytest.raises(ValueError):
            call_store(store, scales(*n), slots)
        with pytest.raises(ValueError):
            call_decode(decode, scales(*n))
    for at in (torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(10, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            call_store(store, scales(3, 2, 4), at)
    with pytest.raises(ValueError):
        fd.make_scales(torch.ones(3, 2, 4), torch.ones(3, 2, 5), block=16)


def test_outputs_have_to_be_as_large_as_the_descriptor_says(fd):  # noqa: F811
    """A 16-bit out under a descriptor for 32 bits (its default) would be written twice over."""
    q, k = torch.zeros(5, 8, 128, dtype=torch.bfloat16), torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    d = fd.make_prompt_desc(q, k, k, batch=0)
    call = lambda out, lse: fd.fd_prompt(d, q, k, k, None, None, out, lse, None, stream=0)
    f32, lse = torch.zeros(5, 8, 128), torch.zeros(5, 8)
    assert call(f32, lse) == call(f32, None) == call(1024, 1024) == fd.FD_OK      # (batch 0: nothing is enqueued)
    for out, z in ((f32.bfloat16(), lse), (f32[:4], lse), (f32.transpose(0, 1), lse), (f32, lse[:4]), (f32, lse.half()),
                   (f32, lse.double()), (f32, lse.t())):
        with pytest.raises(ValueError):
            call(out, z)
    # the other way round: 32 bits under a descriptor for 16
    d = fd.make_prompt_desc(q, k, k, batch=0, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        call(f32, lse)
    assert call(f32.bfloat16(), lse) == fd.FD_OK
    kc = torch.zeros(3, 2, 64, 128).to(torch.float8_e4m3fn)
    s = fd.make_scales(torch.ones(3, 2, 4), torch.ones(3, 2, 4), block=16)
    d = fd.make_desc(q[:3], kc, kc, max_seqlen=64, n_splits=1)
    for out, z in ((f32.bfloat16(), lse), (f32[:2], lse), (f32, lse[:2])):
        with pytest.raises(ValueError):
            fd.fd_decode_scaled(d, s, q, kc, kc, 1024, None, out, z, None, 0, stream=0)


@pytest.mark.parametrize("out_dtype,out,lse,aux", [("f32", 1026, 1024, 1024), ("f16", 1025, 1024, 1024), ("bf16", 1024, 1026, 1024),
                                                   ("f32", 1024, 1024, 1026)])
def test_addresses_are_multiples_of_their_elements(fd, out_dtype, out, lse, aux):  # noqa: F811
    code = {"f32": fd.FD_F32, "f16": fd.FD_F16, "bf16": fd.FD_BF16}[out_dtype]
    d = _prompt(fd)
    d.out_dtype = code
    assert fd.fd_prompt(d, 1024, 1024, 1024, aux, 1024, out, lse, None, 0, stream=0) == fd.FD_ERR_INVALID_ARG
    d = _decode(fd, kv_dtype=fd.FD_E4M3, page_size=64, max_pages_per_seq=4, out_dtype=code)
    assert fd.fd_decode_scaled(d, _scales(fd), 1024, 1024, 1024, aux, 1024, out, lse, 1024, 1 << 30,
                               stream=0) == fd.FD_ERR_INVALID_ARG
    assert fd.fd_decode_scaled(d, _scales(fd), 1024, 1024, 1024, 1024, 1026, 1024, 1024, 1024, 1 << 30,
                               stream=0) == fd.FD_ERR_INVALID_ARG


def test_addresses_are_taken_of_tensors_integers_and_none(fd):  # noqa: F811
    t = torch.zeros(3)
    assert fd._ptr(t) == t.data_ptr() and fd._ptr(1024) == 1024 and fd._ptr(None) is None
    with pytest.raises(TypeError):
        fd._ptr("1024")
