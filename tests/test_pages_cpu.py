"""Refusals and layouts of fd_qkv_rope and of the page operators, checked on the host:
nothing here reaches a GPU.  Addresses are made up; a call that is refused
reads none of them."""
import ctypes

import pytest
import torch

import pages_ref as ref

A = 1 << 20              # an address that nothing reads


@pytest.fixture(scope="module")
def fd():
    import split_kv_gb300
    from split_kv_gb300 import _build
    _build.build()
    return split_kv_gb300


def test_struct_sizes(fd):
    assert ctypes.sizeof(fd.FdRopeDesc) == 14 * 4 + 19 * 8 + 4 * 4
    assert fd.FdRopeDesc.q_stride_t.offset == 56 and fd.FdRopeDesc.page_size.offset == 208
    assert ctypes.sizeof(fd.FdPool) == 48 and fd.FdPool.extent.offset == 32


# ------------------------------------------------------------------ fd_qkv_rope
def rope_desc(fd, **over):
    q, k = torch.zeros(4, 8, 128, dtype=torch.float16), torch.zeros(4, 2, 128, dtype=torch.float16)
    kc = torch.zeros(5, 2, 16, 128, dtype=over.pop("cache", torch.float16))
    d = fd.make_rope_desc(q, k, k, q_out=q, k_out=k, k_cache=kc, v_cache=kc, page_size=16)
    for n, v in over.items():
        setattr(d, n, v)
    return d


def rope_call(fd, d, **over):
    a = dict(q=A, k=A, v=A, q_weight=None, k_weight=None, inv_freq=A, positions=A, slots=A, q_out=2 * A, k_out=2 * A, k_cache=A,
             v_cache=A, stream=0)
    a.update(over)
    return fd.fd_qkv_rope(d, **a)


@pytest.mark.parametrize("over,status", [
    (dict(n_tokens=-1), -1), (dict(n_q_heads=-1), -1), (dict(n_q_heads=0, n_kv_heads=0), -1), (dict(head_dim=64), -2), (dict(head_dim=0), -1),
    (dict(dtype=2), -2), (dict(dtype=3), -2), (dict(dtype=9), -1), (dict(cache_dtype=1), -2), (dict(cache_dtype=9), -1), (dict(w_dtype=3), -2),
    (dict(w_dtype=7), -1), (dict(norm=4), -1), (dict(rot_dim=130), -1), (dict(rot_dim=-2), -1), (dict(rot_dim=15), -1), (dict(rot_dim=24), -2),
    (dict(interleaved=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(rot_scale=float("nan")), -1),
    (dict(q_stride_t=1025), -1), (dict(k_src_stride_h=-8), -1), (dict(q_out_stride_h=64), -1), (dict(q_out_stride_t=0), -1),
    (dict(k_out_stride_t=8), -1), (dict(k_stride_b=0), -1), (dict(v_stride_h=0), -1), (dict(k_stride_t=64), -1), (dict(k_stride_h=4), -1),
    (dict(q_w_stride_h=4), -1), (dict(page_size=12), -1), (dict(page_size=4), -2), (dict(page_size=-8), -1), (dict(page_size=0, batch=0), -1),
    (dict(kv_extent=0), -1), (dict(flags=1), -1), (dict(reserved=1), -1), (dict(n_kv_heads=70000), -2)])
def test_rope_refuses_descriptors(fd, over, status):
    assert rope_call(fd, rope_desc(fd, **over)) == status


@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan"), 1e-40])
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
def test_rope_refuses_scales(fd, name, scale):
    d = rope_desc(fd, cache=torch.float8_e4m3fn)
    setattr(d, name, scale)
    assert rope_call(fd, d) == -1


@pytest.mark.parametrize("over", [
    dict(q=None), dict(k=None), dict(v=None), dict(positions=None), dict(inv_freq=None), dict(slots=None), dict(q_out=None),
    dict(k_cache=None), dict(v_cache=None), dict(k_cache=None, v_cache=None, k_out=None), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4),
    dict(q_out=A + 8), dict(k_out=A + 1), dict(k_cache=A + 8), dict(v_cache=A + 8), dict(positions=A + 2), dict(slots=A + 4), dict(inv_freq=A + 1),
    dict(q_weight=A + 4), dict(k_weight=A + 8)])
def test_rope_refuses_addresses(fd, over):
    assert rope_call(fd, rope_desc(fd), **over) == -1


def test_rope_refuses_in_place_with_other_strides(fd):
    assert rope_call(fd, rope_desc(fd, q_out_stride_t=2048), q_out=A) == -1
    assert rope_call(fd, rope_desc(fd, k_out_stride_t=2048), k_out=A) == -1


def test_rope_of_no_tokens_takes_empty_tensors(fd):
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16)
    d = fd.make_rope_desc(e, e, q_out=e, k_out=e)
    assert fd.fd_qkv_rope(d, e, e, None, None, None, torch.zeros(64), torch.zeros(0, dtype=torch.int32), None, e, e, None, None, 0) == 0


def test_rope_binding_refuses_sizes(fd):
    x = torch.zeros(3, 4, 128, dtype=torch.float16)
    d = fd.make_rope_desc(x, x, q_out=x, k_out=x)
    i, f, s = torch.zeros(3, dtype=torch.int32), torch.zeros(64), torch.zeros(3, dtype=torch.int64)
    for pos, freq, slots in ((i[:2], f, s), (i.long(), f, s), (i.float(), f, s), (i, f[:63], s), (i, f.double(), s), (i, f, s[:2]),
                             (i, f, i), (i, torch.zeros(128)[::2], s), (i, f.int(), s), (i, f, s.double())):
        with pytest.raises(ValueError):
            fd.fd_qkv_rope(d, x, x, None, None, None, freq, pos, slots, x, x, None, None, 0)
    bad = [dict(q=x, k=x.to(torch.bfloat16), q_out=x, k_out=x), dict(q=x, k=x, q_out=x[:2], k_out=x), dict(q=x, k=x, q_out=x),
           dict(q=x, k=x, v=x, q_out=x, k_cache=torch.zeros(2, 4, 16, 128, dtype=torch.float16)),
           dict(q=x, k=x, v=x, q_out=x, k_cache=torch.zeros(2, 3, 16, 128, dtype=torch.float16), v_cache=torch.zeros(2, 3, 16, 128, dtype=torch.float16)),
           dict(q=x, k=x, q_out=x, k_out=x, q_weight=torch.zeros(64)), dict(q=x, k=x, q_out=x, k_out=x, q_weight=torch.zeros(3, 128)),
           dict(q=x, k=x, q_out=x, k_out=x, q_weight=torch.zeros(128), k_weight=torch.zeros(128, dtype=torch.float16))]
    for kw in bad:
        with pytest.raises(ValueError):
            fd.make_rope_desc(kw.pop("q"), kw.pop("k"), kw.pop("v", None), **kw)


# ------------------------------------------------------------------ page operators
def page_desc(fd, **over):
    d = fd.FdPageDesc(batch=4, page_size=16, max_pages_per_seq=8, n_pages=40, n_free_max=40, n_slots=4)
    for n, v in over.items():
        setattr(d, n, v)
    return d


def page_call(fd, op, d, n_forks=2, n_keep=20, **over):
    a = dict(seqlens=A, free_pages=A, free_count=A, block_table=A, shares=A, free_count_out=A, copy_src=A, copy_dst=A, copy_count=A, stream=0)
    if op != "compact":
        a["seqlens_out"] = A
    if op == "fork":
        a.update(parents=A, children=A, keep=None, n_forks=n_forks)
    if op == "trim":
        a["keep"] = A
    if op == "compact":
        a["n_keep"] = n_keep
    a.update(over)
    return getattr(fd, "fd_page_" + op)(d, **a)


@pytest.mark.parametrize("op", ["fork", "trim", "compact"])
@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), -1), (dict(batch=8193), -2), (dict(page_size=0), -1), (dict(page_size=12), -1), (dict(page_size=4), -2),
    (dict(page_size=1 << 21), -1), (dict(max_pages_per_seq=0), -1), (dict(max_pages_per_seq=1 << 28), -1), (dict(n_pages=0), -1),
    (dict(n_free_max=-1), -1), (dict(n_slots=-1), -1)])
def test_pages_refuse_descriptors(fd, op, over, status):
    assert page_call(fd, op, page_desc(fd, **over)) == status


@pytest.mark.parametrize("op,over", [(op, {n: v}) for op, names in (
    ("fork", "parents children seqlens free_pages free_count block_table shares seqlens_out free_count_out copy_src copy_dst copy_count"),
    ("trim", "keep seqlens free_pages free_count block_table seqlens_out free_count_out copy_src copy_dst copy_count"),
    ("compact", "seqlens free_pages free_count block_table free_count_out copy_src copy_dst copy_count")) for n in names.split() for v in (None, A + 2)])
def test_pages_refuse_addresses(fd, op, over):
    assert page_call(fd, op, page_desc(fd), **over) == -1


def test_pages_refuse_counts(fd):
    assert page_call(fd, "fork", page_desc(fd), n_forks=-1) == -1
    assert page_call(fd, "fork", page_desc(fd), n_forks=5) == -1                   # the copy list has 4
    assert page_call(fd, "fork", page_desc(fd, n_slots=9000), n_forks=8193) == -2
    assert page_call(fd, "trim", page_desc(fd, n_slots=3)) == -1
    assert page_call(fd, "trim", page_desc(fd, batch=8192, max_pages_per_seq=1 << 17, n_slots=8192)) == -2
    assert page_call(fd, "compact", page_desc(fd), n_keep=-1) == -1
    assert page_call(fd, "compact", page_desc(fd), n_keep=41) == -1
    assert page_call(fd, "compact", page_desc(fd, n_pages=(1 << 19) + 30), n_keep=29) == -2
    assert page_call(fd, "trim", page_desc(fd), shares=A + 1) == -1


def test_pages_binding_refuses_sizes(fd):
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    table, free, src = i(24).view(3, 8), i(9), i(3)
    with pytest.raises(ValueError):
        fd.make_page_desc(table, free, None, copies=src.long(), page_size=16, n_pages=9)
    with pytest.raises(ValueError):
        fd.make_page_desc(table, free, torch.zeros(3, dtype=torch.int64), copies=src, page_size=16, n_pages=9)
    d = fd.make_page_desc(table, free, None, copies=src, page_size=16, n_pages=9)
    assert (d.batch, d.max_pages_per_seq, d.n_slots, d.n_free_max) == (3, 8, 3, 9)
    good = dict(keep=i(3), seqlens=i(3), free_pages=free, free_count=i(1), block_table=table, shares=i(9), seqlens_out=i(3), free_count_out=i(1),
                copy_src=src, copy_dst=i(3), copy_count=i(1), stream=0)
    for n, v in (("keep", i(2)), ("seqlens", i(3).long()), ("seqlens", i(6)[::2]), ("shares", i(8)), ("seqlens_out", i(2)), ("copy_dst", i(2)),
                 ("copy_dst", i(3).float())):
        with pytest.raises(ValueError):
            fd.fd_page_trim(d, **{**good, n: v})


# ------------------------------------------------------------------ fd_page_copy
def pool(fd, **over):
    x = fd.FdPool(base=A, page_stride=32768, row_bytes=256)
    x.extent[0], x.extent[1], x.stride[0], x.stride[1] = 8, 16, 4096, 256
    for n, v in over.items():
        if isinstance(v, tuple):
            getattr(x, n)[v[0]] = v[1]
        else:
            setattr(x, n, v)
    return x


@pytest.mark.parametrize("over", [
    dict(base=None), dict(row_bytes=0), dict(row_bytes=-1), dict(reserved=1), dict(page_stride=0), dict(page_stride=-16), dict(page_stride=128), dict(page_stride=1 << 39, stride=(0, 1 << 41)),
    dict(page_stride=(1 << 46) // 9 + 1),
    dict(extent=(0, 0)), dict(extent=(1, -1)), dict(stride=(0, 0)), dict(stride=(1, 128)), dict(stride=(0, -4096)), dict(stride=(0, 1 << 41))])
def test_copy_refuses_pools(fd, over):
    two = (fd.FdPool * 2)(pool(fd), pool(fd, **over))
    two.n_pages = 9
    assert fd.fd_page_copy(two, A, A, None, n_pairs=3, stream=0) == -1


def test_copy_refuses_arguments(fd):
    one = (fd.FdPool * 1)(pool(fd))
    one.n_pages = 9
    for src, dst, count, n in ((None, A, None, 3), (A, None, None, 3), (A + 2, A, None, 3), (A, A + 1, None, 3), (A, A, A + 2, 3), (A, A, None, -1)):
        assert fd.fd_page_copy(one, src, dst, count, n_pairs=n, stream=0) == -1
    one.n_pages = 0
    assert fd.fd_page_copy(one, A, A, None, n_pairs=3, stream=0) == -1
    none = fd.make_pools([])
    assert fd.fd_page_copy(none, A, A, None, n_pairs=3, stream=0) == 0


def test_make_pools(fd):
    a = torch.zeros(5, 8, 16, 128, dtype=torch.bfloat16)
    p = fd.make_pools([a, a.permute(0, 2, 1, 3), torch.zeros(5, 8, 2), torch.zeros(5, 3)[:, ::2]])
    assert p.n_pages == 5 and len(p) == 4
    assert (p[0].row_bytes, list(p[0].extent), list(p[0].stride), p[0].page_stride) == (256, [8, 16], [4096, 256], 32768)
    assert (p[1].row_bytes, list(p[1].extent), list(p[1].stride)) == (256, [16, 8], [256, 4096])
    assert (p[2].row_bytes, list(p[2].extent), list(p[2].stride)) == (8, [1, 8], [0, 8])
    assert (p[3].row_bytes, list(p[3].extent), list(p[3].stride), p[3].page_stride) == (4, [1, 2], [0, 8], 12)
    for bad in ([a, a[:4]], [torch.zeros(5, 2, 2, 2, 2, 2)], [torch.zeros(5, 4, 4, 4)[..., ::2]], [torch.zeros(5, 0)]):
        with pytest.raises(ValueError):
            fd.make_pools(bad)


# ------------------------------------------------------------------ the references, by hand
def test_reference_fork_and_trim_by_hand():
    # two sequences of 20 and 0 tokens, pages of 8: pages 3, 1, 5 held, 9, 8, 7 free (7 is taken first)
    out, bad = ref.fork([0], [1], [18], [20, 0], [9, 8, 7], 3, [[3, 1, 5], [0, 0, 0]], [0] * 10, 8, 10, [-1], [-1])
    assert not bad and out["lens"] == [20, 18] and out["table"][1] == [3, 1, 7] and out["count"] == 2
    assert [p for p in range(10) if out["shares"][p]] == [1, 3] and (out["src"], out["dst"], out["n"]) == ([5], [7], 1)
    # both keep 12: page 1 is shared by two that keep a part of it, the last keeps it, the first gets a copy (in 8);
    # then 5 and 7 go back, 5 on top
    back, bad = ref.trim([12, 12], out["lens"], [9, 8, 7], 2, out["table"], out["shares"], 8, 10, [-1, -1], [-1, -1])
    assert not bad and back["table"] == [[3, 8, 5], [3, 1, 7]] and back["src"][0] == 1 and back["dst"][0] == 8
    assert back["count"] == 3 and back["free"] == [9, 7, 5] and back["shares"][1] == 0 and back["shares"][3] == 1
    done, bad = ref.trim([0, 0], back["lens"], back["free"] + [0] * 3, 3, back["table"], back["shares"], 8, 10, [-1, -1], [-1, -1])
    # 3 goes back once, at its last place: 8, 3, 1 in order, 8 on top
    assert not bad and done["count"] == 6 and done["free"] == [9, 7, 5, 1, 3, 8]


def test_reference_compact_by_hand():
    out, bad = ref.compact(4, [16, 9], [8, 0, 2, 9], 4, [[6, 1], [6, 5]], [0, 0, 0, 0, 0, 0, 1, 0, 0, 0], 8, 10, [-1] * 4, [-1] * 4)
    # F = 0, 2; 5 -> 2, 6 -> 0
    assert not bad and out["table"] == [[0, 1], [0, 2]] and out["count"] == 0 and out["n"] == 2
    assert out["src"][:2] == [5, 6] and out["dst"][:2] == [2, 0] and out["shares"][0] == 1 and out["shares"][6] == 0


# ------------------------------------------------------------------ fd_page_tables
def tables_args():
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    return dict(seqlens=i(3), new_tokens=i(3), free_pages=i(9), free_count=i(1), block_table=i(24).view(3, 8), seqlens_out=i(3),
                free_count_out=i(1), cu_tokens=i(4), slots=torch.zeros(6, dtype=torch.int64), positions=i(6), stream=0)


def test_tables_refuse_a_copy_lists_descriptor(fd):
    """Its n_slots is the list's length: slots and positions may be shorter, and would be written behind their ends."""
    a = tables_args()
    for copies in (torch.zeros(100, dtype=torch.int32), torch.zeros(6, dtype=torch.int32), None):
        d = fd.make_page_desc(a["block_table"], a["free_pages"], None, copies=copies, page_size=16, n_pages=9)
        with pytest.raises(ValueError):
            fd.fd_page_tables(d, **a)


def test_tables_binding_refuses_sizes(fd):
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    a = tables_args()
    d = fd.make_page_desc(a["block_table"], a["free_pages"], a["slots"], page_size=16, n_pages=9)
    for n, v in (("seqlens", i(2)), ("seqlens", i(3).long()), ("new_tokens", i(2)), ("new_tokens", i(6)[::2]), ("free_pages", i(8)), ("free_count", i(0)),
                 ("free_count", i(1).long()), ("block_table", i(23)), ("block_table", i(48).view(3, 16)[:, ::2]), ("seqlens_out", i(2)), ("free_count_out", i(0)),
                 ("cu_tokens", i(3)), ("slots", torch.zeros(5, dtype=torch.int64)), ("slots", i(6)), ("positions", i(5)),
                 ("positions", torch.zeros(6, dtype=torch.int64))):
        with pytest.raises(ValueError):
            fd.fd_page_tables(d, **{**a, n: v})
    d.page_size = 4         # (whatever the sizes: refused by the library, so that nothing reaches a GPU here)
    assert fd.fd_page_tables(d, **a) == fd.FD_ERR_UNSUPPORTED
    assert fd.fd_page_tables(d, **{**a, "cu_tokens": None, "positions": None}) == fd.FD_ERR_UNSUPPORTED


# ------------------------------------------------------------------ arrays of the other page calls
@pytest.mark.parametrize("op", ["fork", "trim", "compact"])
def test_page_calls_refuse_arrays_of_other_sizes(fd, op):
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    table, free, src = i(24).view(3, 8), i(9), i(3)
    d = fd.make_page_desc(table, free, None, copies=src, page_size=16, n_pages=9)
    good = dict(seqlens=i(3), free_pages=free, free_count=i(1), block_table=table, shares=i(9), free_count_out=i(1), copy_src=src, copy_dst=i(3),
                copy_count=i(1), stream=0)
    if op == "fork":
        good.update(parents=i(2), children=i(2), keep=None, seqlens_out=i(3))
    elif op == "trim":
        good.update(keep=i(3), seqlens_out=i(3))
    else:
        good["n_keep"] = 4
    call = getattr(fd, "fd_page_" + op)
    bad = [("free_pages", i(8)), ("free_pages", i(9).long()), ("free_count", i(0)), ("free_count", i(1).long()), ("block_table", i(23)),
           ("block_table", table.long()), ("block_table", i(48).view(3, 16)[:, :8]), ("shares", i(8)), ("shares", i(18)[::2]), ("free_count_out", i(0)),
           ("free_count_out", i(1).float()), ("copy_src", i(2)), ("copy_src", i(3).long()), ("copy_dst", i(2)), ("copy_count", i(0)),
           ("copy_count", i(1).long())]
    for n, v in bad:
        with pytest.raises(ValueError):
            call(d, **{**good, n: v})
    d.page_size = 4         # (refused by the library)
    assert call(d, **good) == fd.FD_ERR_UNSUPPORTED


def test_copy_refuses_counts_of_other_types(fd):
    one = (fd.FdPool * 1)(pool(fd))
    one.n_pages = 9
    for count in (torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32), torch.zeros(1)):
        with pytest.raises(ValueError):
            fd.fd_page_copy(one, torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), count, stream=0)


# ------------------------------------------------------------------ tensors of fd_qkv_rope
def test_rope_refuses_weights_that_are_not_its_descriptors(fd):
    """A descriptor without weights says 32 bits: bf16 ones would be read behind their end."""
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    pos, freq, w = torch.zeros(3, dtype=torch.int32), torch.zeros(64), torch.zeros(128, dtype=torch.bfloat16)
    call = lambda d, qw, kw: fd.fd_qkv_rope(d, x, x, None, qw, kw, freq, pos, None, x, x, None, None, 0)
    bare = fd.make_rope_desc(x, x, q_out=x, k_out=x)
    shared = fd.make_rope_desc(x, x, q_out=x, k_out=x, q_weight=w, k_weight=w)
    per_head = fd.make_rope_desc(x, x, q_out=x, k_out=x, q_weight=w.expand(4, 128).clone(), k_weight=w.expand(4, 128).clone())
    for d, qw, kw in ((bare, w, None), (bare, None, w), (bare, torch.zeros(64), None), (shared, w.float(), w), (shared, w, w.half()), (shared, w[:64], w),
                      (per_head, w, None), (per_head, None, torch.zeros(3, 128, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call(d, qw, kw)
    for d in (bare, shared, per_head):
        d.rot_dim = 24              # (refused by the library, so that nothing reaches a GPU here)
    assert call(shared, w, w) == call(shared, w, None) == call(shared, None, None) == call(bare, torch.zeros(128), None) == fd.FD_ERR_UNSUPPORTED
    assert call(per_head, torch.zeros(4, 128, dtype=torch.bfloat16), None) == fd.FD_ERR_UNSUPPORTED
    none = fd.make_rope_desc(x, x, q_out=x, k_out=x, norm_q=False, norm_k=False)
    none.rot_dim = 24
    assert call(none, w, w) == fd.FD_ERR_UNSUPPORTED          # no norm: weights are not read


def test_rope_refuses_tensors_that_are_smaller_than_its_descriptor_says(fd):
    x = torch.zeros(6, 8, 128, dtype=torch.float16)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    pos, freq, slots = torch.zeros(6, dtype=torch.int32), torch.zeros(64), torch.zeros(6, dtype=torch.int64)
    qo, ko = torch.zeros(6, 4, 128, dtype=torch.float16), torch.zeros(6, 2, 128, dtype=torch.float16)
    for page in (16, 0):
        kc, vc = (torch.zeros(5, 2, 16, 128, dtype=torch.float16) for _ in range(2))
        d = fd.make_rope_desc(q, k, v, q_out=qo, k_out=ko, k_cache=kc, v_cache=vc, page_size=page)
        good = dict(q=q, k=k, v=v, q_weight=None, k_weight=None, inv_freq=freq, positions=pos, slots=slots, q_out=qo, k_out=ko, k_cache=kc, v_cache=vc,
                    stream=0)
        for n, t in (("q", q[:5]), ("k", k[:, :1]), ("v", v[1:]), ("q_out", qo[:, :3]), ("k_out", ko[:5]), ("k_cache", kc[:4]),
                     ("v_cache", vc.to(torch.float8_e4m3fn)), ("v_cache", vc[:, :, :8])):
            with pytest.raises(ValueError):
                fd.fd_qkv_rope(d, **{**good, n: t})
        d.rot_dim = 24
        assert fd.fd_qkv_rope(d, **good) == fd.FD_ERR_UNSUPPORTED
        assert fd.fd_qkv_rope(d, **{**good, "k_out": None}) == fd.FD_ERR_UNSUPPORTED
