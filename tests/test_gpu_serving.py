"""The serving operators on the GPU, through the C ABI, against the plain 64-bit
implementations of serving_ref: page tables and the store exactly, the two
attentions within tolerances that follow from their roundings (see there)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import split_kv_gb300 as fd

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from split_kv_gb300 import _build
    _build.build()
    torch.cuda.set_device(DEV)
    fd.fd_device_status(clear=True)
    yield


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert fd.fd_device_status(clear=True) == fd.FD_OK


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, dtype, *shape, gain=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * gain).to(DT[dtype])


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def cumulative(v, first=0):
    out = [first]
    for x in v:
        out.append(out[-1] + x)
    return out


# ------------------------------------------------------------------ page tables
def table_case(seed, batch, page, width, top_new, free=None, extra=5):
    r = np.random.default_rng(seed)
    cap = page * width
    lens = [int(x) for x in r.integers(0, max(1, cap - top_new), size=batch)]
    lens = [x if r.random() < 0.8 else (x // page) * page for x in lens]
    new = [int(x) for x in r.integers(0, top_new + 1, size=batch)]
    have = [-(-x // page) for x in lens]
    need = sum(-(-(a + b) // page) for a, b in zip(lens, new)) - sum(have)
    n_pages = sum(have) + need + 50
    perm = [int(x) for x in r.permutation(n_pages)]
    table, at = [], 0
    for h in have:
        table.append(perm[at:at + h] + [-7] * (width - h))
        at += h
    rest = perm[at:]
    return lens, new, rest, len(rest) if free is None else free, table, n_pages, sum(new) + extra


def run_tables(lens, new, free, count, table, page, n_pages, n_slots, alias=False, batch=None):
    tb = torch.tensor(table, dtype=torch.int32, device=DEV).reshape(len(lens), -1)
    fr = i32(free)
    sl = torch.full((n_slots,), 99, dtype=torch.int64, device=DEV)
    po = torch.full((n_slots,), 99, dtype=torch.int32, device=DEV)
    cu = torch.full((len(lens) + 1,), 99, dtype=torch.int32, device=DEV)
    ln, nw, ct = i32(lens), i32(new), i32([count])
    lo, co = (ln, ct) if alias else (torch.full_like(ln, 99), torch.full_like(ct, 99))
    d = fd.make_page_desc(tb, fr, sl, page_size=page, n_pages=n_pages)
    fd.check(fd.fd_page_tables(d, ln, nw, fr, ct, tb, lo, co, cu, sl, po), "fd_page_tables")
    torch.cuda.synchronize()
    return [lo.tolist(), int(co), tb.tolist(), cu.tolist(), sl.tolist(), po.tolist()]


@pytest.mark.parametrize("batch,page,width,top_new", [
    (1, 16, 40, 1), (1, 8, 3000, 20000), (5, 16, 64, 700), (64, 16, 300, 1), (33, 128, 20, 500), (257, 32, 30, 40),
    (1025, 64, 6, 9), (3000, 16, 4, 2), (8192, 8, 3, 3)])
@pytest.mark.parametrize("alias", [False, True])
def test_tables(batch, page, width, top_new, alias):
    lens, new, free, count, table, n_pages, n_slots = table_case(batch * 7 + page, batch, page, width, top_new)
    want = ref.tables(lens, new, free, count, table, page, n_pages, n_slots)
    got = run_tables(lens, new, free, count, table, page, n_pages, n_slots, alias)
    for name, a, b in zip(("lens", "count", "table", "cu", "slots", "positions"), got, want):
        assert a == b, name
    assert not want[6]


@pytest.mark.parametrize("what", ["few pages", "no pages", "few slots", "long", "negative length", "negative count",
                                  "bad free page", "bad table entry", "free count"])
def test_tables_report_what_does_not_fit(what):
    page, width = 16, 30
    lens, new, free, count, table, n_pages, n_slots = table_case(11, 9, page, width, 120)
    new[4] = max(new[4], 17)
    lens[2], new[2] = 33, 5                        # goes on in a page it has
    table[2] = [1, 2, 3] + [-7] * (width - 3)
    if what == "few pages":
        count = 9
    elif what == "no pages":
        count = 0
    elif what == "few slots":
        n_slots = sum(new[:5]) + 1
    elif what == "long":
        lens[3] = page * width - 3
        new[3] = 4
        table[3] = [4] * width
        n_slots += 4
    elif what == "negative length":
        lens[3] = -1
    elif what == "negative count":
        new[3] = -5
    elif what == "bad free page":
        free[count - 2] = n_pages
    elif what == "bad table entry":
        table[2][2] = -1
    else:
        count = len(free) + 1
    want = ref.tables(lens, new, free, count, table, page, n_pages, n_slots)
    got = run_tables(lens, new, free, count, table, page, n_pages, n_slots)
    for name, a, b in zip(("lens", "count", "table", "cu", "slots", "positions"), got, want):
        assert a == b, name
    assert want[6] and fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS


def test_tables_advance_in_a_captured_graph():
    """A decode step's tables captured once, lengths and free count in place."""
    page, width, batch = 16, 8, 5
    lens, table = [0, 15, 16, 31, 100], []
    perm = [int(x) for x in np.random.default_rng(3).permutation(60)]
    at = 0
    for x in lens:
        h = -(-x // page)
        table.append(perm[at:at + h] + [-7] * (width - h))
        at += h
    free = perm[at:]
    tb, fr, ln, ct = i32(table), i32(free), i32(lens), i32([len(free)])
    sl = torch.zeros(batch, dtype=torch.int64, device=DEV)
    d = fd.make_page_desc(tb, fr, sl, page_size=page, n_pages=60)
    one = i32([1] * batch)

    def step():
        fd.check(fd.fd_page_tables(d, ln, one, fr, ct, tb, ln, ct, None, sl, None))

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    want = (lens, len(free), table)
    for k in range(20):
        if k > 0:
            g.replay()
        w = ref.tables(want[0], [1] * batch, free, want[1], want[2], page, 60, batch)
        assert [ln.tolist(), int(ct), tb.tolist(), sl.tolist()] == [w[0], w[1], w[2], w[4]]
        want = w[:3]


# ------------------------------------------------------------------ store
def store_case(seed, dtype, lens, held, H, page, block, gain=1.0, contiguous=0, hnd=True):
    g = gen(seed)
    B = len(lens)
    if contiguous:
        lead, tok = B, contiguous
        slots = torch.cat([torch.arange(h, h + n, device=DEV) + b * contiguous for b, (h, n) in enumerate(zip(held, lens))])
    else:
        tok = page
        width = max(-(-(h + n) // page) for h, n in zip(held, lens))
        lead = B * width + 3
        table = torch.randperm(lead, generator=g, device=DEV)[:B * width].view(B, width)
        slots = torch.cat([table[b, torch.arange(h, h + n, device=DEV) // page] * page
                           + torch.arange(h, h + n, device=DEV) % page for b, (h, n) in enumerate(zip(held, lens))])
    nb = -(-tok // block)
    caches, scales = [], []
    for _ in range(2):
        x = torch.randint(0, 256, (lead, tok, H, D), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        x = torch.where((x & 0x7f) == 0x7f, torch.zeros_like(x), x).view(ref.F8)
        caches.append(x.permute(0, 2, 1, 3).contiguous() if hnd else x.permute(0, 2, 1, 3))
        scales.append(torch.exp2(torch.randint(-12, -4, (lead, H, nb), generator=g, device=DEV).float()))
    n = sum(lens)
    k, v = randn(g, dtype, n, H, D, gain=gain), randn(g, dtype, n, H, D, gain=gain)
    # a wide spread between rows, so that scales grow inside a block
    k *= torch.exp2(torch.randint(-6, 7, (n, 1, 1), generator=g, device=DEV).float()).to(k.dtype)
    return k, v, slots, caches, scales


def bits(x):
    return x.contiguous().view(torch.uint8)


def run_store(k, v, slots, caches, scales, page, block):
    want = [ref.store(x, slots, c, s, page or c.shape[2], block) for x, c, s in zip((k, v), caches, scales)]
    sc = fd.make_scales(*scales, block=block)
    d = fd.make_store_desc(k, v, *caches, page_size=page)
    fd.check(fd.fd_cache_store(d, sc, k, v, slots, *caches), "fd_cache_store")
    torch.cuda.synchronize()
    for name, c, s, (wc, ws) in zip("kv", caches, scales, want):
        assert torch.equal(s.double(), ws), f"{name} scales"
        got = c.double()
        same = (got == wc) | (torch.isnan(got) & torch.isnan(wc))
        assert bool(same.all()), f"{name}: {int((~same).sum())} values differ"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 64), (64, 16), (128, 32), (8, 8), (16, 1), (1024, 1024)])
@pytest.mark.parametrize("lens,held", [([1], [0]), ([1, 1, 1], [5, 16, 31]), ([200, 1, 37, 64, 130], [0, 63, 3, 64, 127]),
                                       ([1500], [17])])
def test_store(dtype, page, block, lens, held):
    run_store(*store_case(page + block + len(lens), dtype, lens, held, 3, page, block), page, block)


@pytest.mark.parametrize("hnd", [False, True])
def test_store_contiguous_cache_with_a_ragged_last_block(hnd):
    # 100 tokens per sequence, blocks of 32: sequence b ends inside a block and b + 1 follows it in the slots
    case = store_case(5, "bf16", [100, 60, 1], [0, 40, 99], 2, 0, 32, contiguous=100, hnd=hnd)
    run_store(*case, 0, 32)


def test_store_page_major_cache_and_strided_rows():
    k, v, slots, caches, scales = store_case(6, "f16", [70, 3], [2, 9], 4, 32, 16, hnd=False)
    fused = torch.cat([k, v], 1)                   # [n, 2H, D]: rows of one projection
    run_store(fused[:, :4], fused[:, 4:], slots, caches, scales, 32, 16)


def test_store_skips_negative_slots_and_flags_those_outside():
    k, v, slots, caches, scales = store_case(7, "bf16", [20, 5], [0, 3], 2, 16, 16)
    slots[3] = -1
    slots[21] = -5
    run_store(k, v, slots, caches, scales, 16, 16)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    slots[7] = caches[0].shape[0] * 16
    slots[22] = 1 << 40
    run_store(k, v, slots, caches, scales, 16, 16)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_store_special_values(dtype):
    """Zeros, subnormals, infinities, NaN, the type's largest value and 7 * 2^k (448 s exactly)."""
    k, v, slots, caches, scales = store_case(8, dtype, [64], [0], 2, 16, 16)
    t = DT[dtype]
    k[0:16] = 0
    k[16:32, 0] = torch.finfo(t).tiny / 8
    k[17, 1, 5] = float("inf")
    k[18, 1, 6] = -float("inf")
    k[19, 1, 7] = NAN
    v[0:16] = 0
    v[3, 0, 0] = 7.0
    v[4, 1, 0] = -torch.finfo(t).max
    v[16:32] = NAN
    run_store(k, v, slots, caches, scales, 16, 16)


def test_store_one_token_at_a_time_equals_the_running_rule():
    """40 single-row calls, growing magnitudes: each block's scale grows and its rows are rewritten."""
    k, v, slots, caches, scales = store_case(9, "bf16", [40], [0], 2, 64, 32)
    k *= torch.exp2(torch.arange(40, device=DEV).float() / 3)[:, None, None].to(k.dtype)
    wc, ws = caches[0].double(), scales[0].double()
    sc = fd.make_scales(*scales, block=32)
    for t in range(40):
        rows = k[t:t + 1], v[t:t + 1]
        wc, ws = ref.store(rows[0], slots[t:t + 1], wc, ws, 64, 32)
        d = fd.make_store_desc(*rows, *caches, page_size=64)
        fd.check(fd.fd_cache_store(d, sc, *rows, slots[t:t + 1].clone(), *caches))
    torch.cuda.synchronize()
    assert torch.equal(scales[0].double(), ws) and torch.equal(caches[0].double(), wc)


# ------------------------------------------------------------------ decode over the scaled cache
def scaled_case(seed, dtype, lens, q_len, hq, hkv, page, block, spread=2, T=None):
    g = gen(seed)
    B = len(lens)
    q = randn(g, dtype, B, q_len, hq, D)
    if page:
        width = max(1, max(-(-n // page) for n in lens))
        lead, tok = B * width + 2, page
        table = torch.randperm(lead, generator=g, device=DEV)[:B * width].view(B, width).to(torch.int32)
    else:
        lead, tok, table = B, T or max(1, max(lens)), None
    nb = -(-tok // block)
    caches, scales = [], []
    for _ in range(2):
        x = (torch.randn(lead, hkv, tok, D, generator=g, device=DEV) * 100).clamp(-448, 448).to(ref.F8)
        caches.append(x)
        scales.append(torch.rand(lead, hkv, nb, generator=g, device=DEV) * 0.01
                      * torch.exp2(torch.randint(-spread, spread + 1, (lead, hkv, nb), generator=g, device=DEV).float()) + 1e-4)
    return q, caches, scales, table


def run_scaled(q, caches, scales, table, lens, page, block, out_dtype=torch.float32, n_splits=0, k_scale=1.0,
               v_scale=1.0, stream=None):
    B, ql, hq, _ = q.shape
    sl = i32(list(lens))
    d = fd.make_desc(q, *caches, page_size=page, max_pages_per_seq=table.shape[1] if table is not None else 0,
                     max_seqlen=max(lens), out_dtype=out_dtype, n_splits=n_splits, k_scale=k_scale, v_scale=v_scale)
    out = torch.full((B, ql, hq, D), NAN, dtype=out_dtype, device=DEV)
    lse = torch.full((B, ql, hq), NAN, device=DEV)
    ws = torch.empty(fd.fd_workspace_size(d), dtype=torch.uint8, device=DEV)
    fd.check(fd.fd_decode_scaled(d, fd.make_scales(*scales, block=block), q, *caches, sl, table, out, lse, ws,
                                 stream=stream), "fd_decode_scaled")
    torch.cuda.synchronize()
    return out, lse


def check_scaled(q, caches, scales, table, lens, page, block, out_dtype=torch.float32, what="", **kw):
    out, lse = run_scaled(q, caches, scales, table, lens, page, block, out_dtype, **kw)
    kw.pop("n_splits", None)
    o, z, tol, ltol = ref.decode(q, *caches, *scales, block, lens, table, page, out_dtype, **kw)
    ref.close(out, o, tol, what + " out")
    ref.close(lse, z, ltol, what + " lse")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("page,block", [(0, 64), (16, 16), (64, 16), (128, 128), (8, 4), (32, 1), (0, 1024)])
@pytest.mark.parametrize("q_len,G", [(1, 1), (1, 4), (1, 8), (4, 4), (3, 7), (1, 40)])
def test_scaled_decode(dtype, page, block, q_len, G):
    lens = [1, 700, 0, 96, 1111]
    case = scaled_case(page + block + G, dtype, lens, q_len, 2 * G, 2, page, block)
    check_scaled(*case, lens, page, block)


@pytest.mark.parametrize("n_splits", [1, 2, 7, 33, 128])
@pytest.mark.parametrize("out_dtype", ["f32", "f16", "bf16"])
def test_scaled_decode_splits_and_outputs(n_splits, out_dtype):
    lens = [4097, 333]
    case = scaled_case(n_splits, "bf16", lens, 1, 16, 4, 64, 32)
    check_scaled(*case, lens, 64, 32, DT[out_dtype], n_splits=n_splits, k_scale=-0.5, v_scale=3.0)


def test_scaled_decode_two_splits_per_cta():
    """More splits than SMs in one wave: the CTA that serves two."""
    lens = [20000]
    S = 2 * fd.fd_num_sms() // 8
    case = scaled_case(3, "f16", lens, 1, 32, 8, 0, 64)
    check_scaled(*case, lens, 0, 64, n_splits=min(S, 128))


def test_scaled_decode_wide_scale_ranges_and_zero_blocks():
    """Scales from 2^-20 to 2^20 beside each other, blocks of scale 0, scores in the hundreds."""
    lens = [3000, 2999]
    q, caches, scales, table = scaled_case(4, "f16", lens, 1, 8, 2, 16, 16, spread=4)
    for s in scales:
        s[::3, :, 0] *= 2.0 ** 10
        s[1::3, :, 0] *= 2.0 ** -10
    scales[1][::2] *= 2.0 ** 10
    scales[1][5::7] = 0
    scales[0][::5] = 0
    check_scaled(q, caches, scales, table, lens, 16, 16)


@pytest.mark.parametrize("page", [0, 16, 64])
def test_scaled_decode_ignores_what_lies_past_the_end(page):
    """NaN bytes and NaN / infinite scales behind each sequence's last token."""
    lens, block = [5, 100, 48, 33], 16
    q, caches, scales, table = scaled_case(5, "bf16", lens, 1, 8, 2, page, block, T=200)
    for x, s in zip(caches, scales):
        for b, n in enumerate(lens):
            tok = x.shape[2]
            if page:
                last = int(table[b, n // page]) if n // page < table.shape[1] else None
                for j in range(-(-n // page), table.shape[1]):
                    x[int(table[b, j])].view(torch.uint8).fill_(0x7f)
                    s[int(table[b, j])] = NAN
                if last is not None and n % page:
                    x[last, :, n % page:].view(torch.uint8).fill_(0x7f)
                    s[last, :, -(-(n % page) // block):] = float("inf")
            else:
                x[b, :, n:].view(torch.uint8).fill_(0x7f)
                s[b, :, -(-n // block):] = NAN
    clean = [torch.nan_to_num(s, 1.0, 1.0) for s in scales]
    out, lse = run_scaled(q, caches, scales, table, lens, page, block)
    kc = [torch.where((c.view(torch.uint8) & 0x7f) == 0x7f, 0, c.view(torch.uint8)).view(ref.F8) for c in caches]
    o, z, tol, ltol = ref.decode(q, *kc, *clean, block, lens, table, page, torch.float32)
    ref.close(out, o, tol, "out")
    ref.close(lse, z, ltol, "lse")


def test_scaled_decode_flags_bad_pages_and_lengths():
    lens = [100, 64]
    q, caches, scales, table = scaled_case(6, "f16", lens, 1, 8, 2, 16, 16)
    table[0, 2] = caches[0].shape[0] + 5
    run_scaled(q, caches, scales, table, lens, 16, 16)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS
    table[0, 2] = 0
    run_scaled(q, caches, scales, table, [-3, 10000], 16, 16)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS


def test_scaled_decode_with_unit_scales_equals_fd_decode():
    """Scales of 1: the same weights as the unscaled kernel's, so nearly its result."""
    lens = [4000, 77]
    q, caches, scales, table = scaled_case(7, "f16", lens, 1, 32, 8, 64, 64)
    for s in scales:
        s.fill_(1.0)
    out, lse = run_scaled(q, caches, scales, table, lens, 64, 64, k_scale=0.01, v_scale=0.01)
    d = fd.make_desc(q, *caches, page_size=64, max_pages_per_seq=table.shape[1], max_seqlen=4000, k_scale=0.01, v_scale=0.01)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(fd.fd_workspace_size(d), dtype=torch.uint8, device=DEV)
    fd.check(fd.fd_decode(d, q, *caches, i32(lens), table, o2, l2, ws))
    torch.cuda.synchronize()
    # both differ from the exact result by at most the reference's tolerance
    o, z, tol, ltol = ref.decode(q, *caches, *scales, 64, lens, table, 64, torch.float32, 0.01, 0.01)
    ref.close(out, o2, 2 * tol, "out")
    ref.close(lse, l2, 2 * ltol, "lse")


# ------------------------------------------------------------------ prompts
def prompt_case(seed, dtype, lens, keys, hq, hkv, gain=1.0, lead=0, tail=0):
    """Packed inputs with `lead` rows before and `tail` rows behind the sequences."""
    g = gen(seed)
    tq, tk = lead + sum(lens) + tail, lead + sum(keys) + tail
    q = randn(g, dtype, tq, hq, D, gain=gain)
    k, v = randn(g, dtype, tk, hkv, D), randn(g, dtype, tk, hkv, D)
    return q, k, v, cumulative(lens, lead), cumulative(keys, lead)


def run_prompt(q, k, v, cq, ck, causal, out_dtype=torch.float32, n_splits=0, fill=NAN, stream=None):
    d = fd.make_prompt_desc(q, k, v, batch=len(cq) - 1, causal=causal, out_dtype=out_dtype, n_splits=n_splits)
    out = torch.full(q.shape, fill, dtype=out_dtype, device=DEV)
    lse = torch.full(q.shape[:2], fill, device=DEV)
    size = fd.fd_prompt_workspace_size(d)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV) if size else None
    fd.check(fd.fd_prompt(d, q, k, v, i32(cq), i32(ck), out, lse, ws, stream=stream), "fd_prompt")
    torch.cuda.synchronize()
    return out, lse


def check_prompt(q, k, v, cq, ck, causal, out_dtype=torch.float32, **kw):
    out, lse = run_prompt(q, k, v, cq, ck, causal, out_dtype, **kw)
    o, z, tol, ltol = ref.prompt(q, k, v, cq, ck, causal, out_dtype)
    ref.close(out, o, tol, "out")                  # NaN stays in the rows of no sequence
    ref.close(lse, z, ltol, "lse")


@pytest.mark.parametrize("n", [1, 2, 63, 127, 128, 129, 255, 256, 257, 511, 640, 1000])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (3, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_lengths(n, hq, hkv, causal):
    check_prompt(*prompt_case(n, "bf16", [n], [n], hq, hkv), causal)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("out_dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (5, 1), (12, 4), (1, 1)])
def test_prompt_packed_types_and_heads(dtype, out_dtype, hq, hkv):
    lens = [300, 1, 17, 129, 512, 64]
    check_prompt(*prompt_case(hq, dtype, lens, lens, hq, hkv), True, DT[out_dtype])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (2, 2)])
def test_prompt_keys_and_queries_of_different_numbers(causal, hq, hkv):
    """Keys that are there already, rows without keys, sequences without queries or keys; rows of no sequence stay."""
    lens = [100, 300, 1, 0, 130, 200, 40]
    keys = [900, 300, 700, 50, 0, 70, 41]
    check_prompt(*prompt_case(2, "f16", lens, keys, hq, hkv, lead=3, tail=70), causal)


def test_prompt_many_sequences():
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 90, size=150)]
    check_prompt(*prompt_case(3, "bf16", lens, lens, 4, 4), True)


def test_prompt_long():
    check_prompt(*prompt_case(4, "bf16", [5000], [5000], 2, 1), True)
    check_prompt(*prompt_case(5, "f16", [200], [9000], 2, 1), True)


@pytest.mark.parametrize("n_splits", [2, 3, 8])
def test_prompt_splits(n_splits):
    lens, keys = [100, 300, 1, 130, 0, 200], [900, 300, 700, 0, 30, 70]
    check_prompt(*prompt_case(6, "bf16", lens, keys, 4, 2, lead=2, tail=9), True, n_splits=n_splits)
    check_prompt(*prompt_case(7, "f16", lens, keys, 3, 3), False, torch.float16, n_splits=n_splits)


def test_prompt_planned_splits():
    """Few queries over long keys: the plan cuts the keys, and asks for a workspace."""
    q, k, v, cq, ck = prompt_case(14, "bf16", [70, 1, 20], [6000, 900, 20], 6, 2, lead=1, tail=3)
    d = fd.make_prompt_desc(q, k, v, batch=3, max_k=6000)
    assert fd.fd_prompt_workspace_size(d) > 0
    check_prompt(q, k, v, cq, ck, True)
    check_prompt(q, k, v, cq, ck, False, torch.bfloat16)
    out = torch.zeros(q.shape, device=DEV)
    assert fd.fd_prompt(d, q, k, v, i32(cq), i32(ck), out, None, None) == fd.FD_ERR_WORKSPACE


def test_prompt_large_scores_move_the_reference():
    """Scores in the hundreds that grow along the keys, so that O is rescaled again and again."""
    q, k, v, cq, ck = prompt_case(8, "f16", [700], [700], 4, 2, gain=6.0)
    k *= torch.linspace(0.1, 3.0, 700, device=DEV)[:, None, None].half()
    check_prompt(q, k, v, cq, ck, True)
    check_prompt(q, k, v, cq, ck, False)


def test_prompt_slices_of_one_projection():
    g = gen(9)
    lens = [250, 131]
    qkv = randn(g, "bf16", sum(lens), 8 + 2 * 2, D)
    check_prompt(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], cumulative(lens), cumulative(lens), True)


def test_prompt_heads_before_rows():
    g = gen(10)
    q, k, v = randn(g, "f16", 8, 300, D), randn(g, "f16", 4, 300, D), randn(g, "f16", 4, 300, D)
    check_prompt(q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), [0, 300], [0, 300], True)


def test_prompt_unaligned_output():
    q, k, v, cq, ck = prompt_case(11, "bf16", [140], [140], 2, 2)
    buf = torch.full((140 * 2 * D + 1,), NAN, dtype=torch.bfloat16, device=DEV)
    d = fd.make_prompt_desc(q, k, v, batch=1, out_dtype=torch.bfloat16)
    fd.check(fd.fd_prompt(d, q, k, v, i32(cq), i32(ck), buf[1:], None))
    torch.cuda.synchronize()
    want, _ = run_prompt(q, k, v, cq, ck, True, torch.bfloat16)
    assert torch.equal(buf[1:].view_as(want), want)


@pytest.mark.parametrize("n_splits", [1, 3])
@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_prompt_special_values_reach_only_who_sees_them(value, n_splits):
    """In K and V of padding rows, of the next sequence, and of a later key of the same sequence."""
    lens = [300, 200]
    q, k, v, cq, ck = prompt_case(12, "bf16", lens, lens, 4, 2, tail=100)
    k[500:], v[500:] = value, value
    check_prompt(q, k, v, cq, ck, True, n_splits=n_splits)
    o0, l0 = run_prompt(q, k, v, cq, ck, True, n_splits=n_splits)
    v[170, 0, 7] = value                           # seen by queries 170.. of sequence 0, heads 0 and 1
    o1, l1 = run_prompt(q, k, v, cq, ck, True, n_splits=n_splits)
    hit = torch.zeros_like(o1, dtype=torch.bool)
    hit[170:300, 0:2, 7] = True
    assert not bool(torch.isfinite(o1[hit]).any())
    o, z, tol, ltol = ref.prompt(q, k, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), cq, ck, True, torch.float32)
    ok = ~hit & torch.isfinite(o)
    assert bool(((o1.double() - o).abs()[ok] <= 2 * tol[ok]).all())
    ref.close(l1, z, ltol, "lse")
    v[170, 0, 7] = 0
    k[260, 1, 3] = NAN                             # scores of key 260 for heads 2 and 3
    o2, l2 = run_prompt(q, k, v, cq, ck, True, n_splits=n_splits)
    assert bool(torch.isnan(o2[260:300, 2:]).all()) and bool(torch.isnan(l2[260:300, 2:]).all())
    assert bool(torch.isfinite(o2[:260]).all()) and bool(torch.isfinite(o2[:300, :2]).all())


def test_prompt_flags_bad_offsets_and_runs_the_rest():
    lens = [100, 50, 70]
    q, k, v, cq, ck = prompt_case(13, "f16", lens, lens, 2, 1)
    want, _ = run_prompt(q, k, v, cq, ck, True)
    bad = list(ck)
    bad[3] = 10000                                 # sequence 2 would read past k
    out, lse = run_prompt(q, k, v, cq, bad, True)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS
    assert torch.equal(out[:150], want[:150]) and bool(torch.isnan(out[150:]).all())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_decode_steps_through_the_scaled_cache(captured):
    """Tables, prompt attention and store of three requests, then decode steps
    (tables, store, scaled decode; captured into one graph or not) on a side
    stream: each step against the plain attention over what the cache holds."""
    hq, hkv, page, block, steps = 8, 2, 16, 16, 12
    lens = [37, 200, 1]
    g = gen(21)
    pool = 60
    tb = torch.full((3, 20), -1, dtype=torch.int32, device=DEV)
    fr, ct, ln = torch.randperm(pool, generator=g, device=DEV).to(torch.int32), i32([pool]), i32([0, 0, 0])
    kc, vc = (torch.zeros(pool, hkv, page, D, device=DEV).to(ref.F8) for _ in range(2))
    ks, vs = (torch.ones(pool, hkv, page // block, device=DEV) for _ in range(2))
    sc = fd.make_scales(ks, vs, block=block)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n = sum(lens)
        q, k, v = randn(g, "bf16", n, hq, D), randn(g, "bf16", n, hkv, D), randn(g, "bf16", n, hkv, D)
        sl = torch.zeros(n, dtype=torch.int64, device=DEV)
        pd = fd.make_page_desc(tb, fr, sl, page_size=page, n_pages=pool)
        fd.check(fd.fd_page_tables(pd, ln, i32(lens), fr, ct, tb, ln, ct, cu, sl, None))
        out = torch.zeros_like(q)
        fd.check(fd.fd_prompt(fd.make_prompt_desc(q, k, v, batch=3, out_dtype=torch.bfloat16), q, k, v, cu, cu, out, None))
        fd.check(fd.fd_cache_store(fd.make_store_desc(k, v, kc, vc, page_size=page), sc, k, v, sl, kc, vc))
        side.synchronize()
        o, _, tol, _ = ref.prompt(q, k, v, cumulative(lens), cumulative(lens), True, torch.bfloat16)
        ref.close(out, o, tol, "prompt")
        assert ln.tolist() == lens
        q1, k1, v1 = randn(g, "bf16", 3, hq, D), randn(g, "bf16", 3, hkv, D), randn(g, "bf16", 3, hkv, D)
        one, sl1 = i32([1, 1, 1]), torch.zeros(3, dtype=torch.int64, device=DEV)
        pd1 = fd.make_page_desc(tb, fr, sl1, page_size=page, n_pages=pool)
        sd1 = fd.make_store_desc(k1, v1, kc, vc, page_size=page)
        dd = fd.make_desc(q1, kc, vc, page_size=page, max_pages_per_seq=20, max_seqlen=320)
        o1, l1 = torch.zeros(3, hq, D, device=DEV), torch.zeros(3, hq, device=DEV)
        ws = torch.empty(fd.fd_workspace_size(dd), dtype=torch.uint8, device=DEV)

        def step():
            fd.check(fd.fd_page_tables(pd1, ln, one, fr, ct, tb, ln, ct, None, sl1, None))
            fd.check(fd.fd_cache_store(sd1, sc, k1, v1, sl1, kc, vc))
            fd.check(fd.fd_decode_scaled(dd, sc, q1, kc, vc, ln, tb, o1, l1, ws))

        graph = None
        if captured:
            keep = [x.clone() for x in (tb, ct, ln, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
            step()
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
            for x, y in zip((tb, ct, ln, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), keep):
                x.copy_(y)
        rows = [k.clone(), v.clone()]
        for s in range(steps):
            for x in (q1, k1, v1):
                x.copy_(torch.randn(x.shape, generator=g, device=DEV) * 1.2 ** s)
            graph.replay() if captured else step()
            side.synchronize()
            now = [n + s + 1 for n in lens]
            assert ln.tolist() == now
            o, z, tol, ltol = ref.decode(q1[:, None], kc, vc, ks, vs, block, now, tb, page, torch.float32)
            ref.close(o1[:, None], o, tol, f"step {s} out")
            ref.close(l1[:, None], z, ltol, f"step {s} lse")
            # what the cache holds for the newest token: within half a step of its block's grid
            for b in range(3):
                pg, off = int(tb[b, (now[b] - 1) // page]), (now[b] - 1) % page
                got = kc[pg, :, off].double() * ks[pg, :, off // block].double()[:, None]
                err = (got - k1[b].double()).abs()
                assert bool((err <= k1[b].double().abs() * 2.0 ** -4 + ks[pg, :, off // block].double()[:, None] * 2.0 ** -10).all())
