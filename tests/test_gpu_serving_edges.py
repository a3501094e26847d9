"""The serving operators at the edges of what their calls allow: batches around
the shared-memory limit, empty steps, many infinities, several threads."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import serving_ref as ref
import split_kv_gb300 as fd
from test_gpu_serving import (DEV, NAN, D, _clean_status, _lib, check_scaled, gen, i32,  # noqa: F401
                              prompt_case, randn, run_prompt, run_scaled, run_store, run_tables,
                              scaled_case, store_case, table_case)

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


# ------------------------------------------------------------------ page tables
def check_tables(batch, page=16, width=4, top_new=2):
    case = table_case(batch, batch, page, width, top_new)
    lens, new, free, count, table, n_pages, n_slots = case
    want = ref.tables(lens, new, free, count, table, page, n_pages, n_slots)
    got = run_tables(lens, new, free, count, table, page, n_pages, n_slots)
    for name, a, b in zip(("lens", "count", "table", "cu", "slots", "positions"), got, want):
        assert a == b, (batch, name)


def test_tables_around_the_default_shared_memory_limit():
    """3 * 4 batch + 4 bytes of dynamic and 272 of static shared memory pass 48 KB
    from batch 4074 on.  A process of its own: no larger batch has been there before."""
    code = ("import sys; sys.path.insert(0, %r); sys.path.insert(0, %r); import torch, test_gpu_serving_edges as t\n"
            "for b in (4073, 4074, 4095, 4096, 8192): t.check_tables(b)\n"
            "assert t.fd.fd_device_status() == 0; print('fine')" % (HERE, os.path.dirname(HERE)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_tables_of_two_threads_with_batches_of_different_sizes():
    cases = {b: table_case(b, b, 16, 4, 2) for b in (4200, 8000)}
    want = {b: ref.tables(*c[:5], 16, c[5], c[6]) for b, c in cases.items()}
    failed = []

    def work(b):
        lens, new, free, count, table, n_pages, n_slots = cases[b]
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = run_tables(lens, new, free, count, table, 16, n_pages, n_slots)
                    assert all(x == y for x, y in zip(got, want[b]))
        except Exception as e:                     # a thread's failure is the test's
            failed.append(f"{b}: {e!r}"[:500])

    threads = [threading.Thread(target=work, args=(b,)) for b in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# ------------------------------------------------------------------ the status word
def test_status_keeps_bits_of_every_operator_until_cleared():
    """Bits that the page tables, the store and the prompt attention raised are joined, and stay where a read does not clear."""
    lens, new, free, count, table, n_pages, n_slots = table_case(3, 4, 16, 8, 20)
    k = randn(gen(1), "f16", 1, 2, D)
    cache = [torch.zeros(3, 2, 16, D, device=DEV).to(ref.F8) for _ in range(2)]
    scales = [torch.ones(3, 2, 1, device=DEV) for _ in range(2)]
    q, pk, pv, cq, ck = prompt_case(1, "f16", [20], [20], 2, 1)
    raisers = (lambda: run_tables(lens, new, free, len(free) + 1, table, 16, n_pages, n_slots),
               lambda: fd.check(fd.fd_cache_store(fd.make_store_desc(k, k, *cache, page_size=16), fd.make_scales(*scales, block=16),
                                                  k, k, torch.tensor([48], device=DEV), *cache)),
               lambda: run_prompt(q, pk, pv, cq, [0, 21], True))
    for some in ((0,), (1,), (2,), (0, 1, 2)):
        for i in some:
            raisers[i]()
        for _ in range(2):
            assert fd.fd_device_status(clear=False) == fd.FD_ERR_DEVICE_BOUNDS
        assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS
        assert fd.fd_device_status(clear=True) == fd.FD_OK


# ------------------------------------------------------------------ prompts with many infinities
@pytest.mark.parametrize("n_splits", [1, 3])
@pytest.mark.parametrize("where,value", [("third", NAN), ("late", NAN), ("all", NAN), ("all", float("inf")),
                                         ("dims", -float("inf")), ("mixed", None)])
def test_prompt_many_special_values(where, value, n_splits):
    """A few thousand keys of which many have infinities or NaN in V: results as
    the definition's, and no wait of the kernel runs out however many rows are
    computed again.  (bf16: no weight of these scores rounds to 0, so that an
    infinity times its weight stays one.)"""
    n = 3000 if where != "dims" else 2200
    q, k, v, cq, ck = prompt_case(31, "bf16", [n, 200], [n + 70, 200], 4, 2)
    if where == "third":
        v[1000::3] = value
    elif where == "late":
        v[n // 2 + 5:, :, ::2] = value
    elif where == "all":
        v[:] = value
    elif where == "dims":                          # another first one in every dim
        for d in range(D):
            v[17 * d + 11, :, d] = value
    else:
        g = gen(32)
        at = torch.randint(0, v.numel(), (400,), generator=g, device=DEV)
        kinds = torch.tensor([NAN, float("inf"), -float("inf")], device=DEV, dtype=v.dtype)
        v.view(-1)[at] = kinds[torch.randint(0, 3, (400,), generator=g, device=DEV)]
    out, lse = run_prompt(q, k, v, cq, ck, True, n_splits=n_splits)
    clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    o, z, tol, ltol = ref.prompt(q, k, clean, cq, ck, True, torch.float32)
    ref.close(lse, z, ltol, "lse")
    # which results are NaN or infinite by right: what kinds of values each row sees in each dim
    for b in range(2):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        seen = torch.arange(nq, device=DEV) + nk - nq
        for h in range(4):
            vv, got = v[ck[b]:ck[b + 1], h // 2], out[cq[b]:cq[b + 1], h].double()
            some = [x.cummax(0).values[seen] for x in (torch.isnan(vv).byte(), (vv == float("inf")).byte(), (vv == -float("inf")).byte())]
            nan = (some[0] | (some[1] & some[2])).bool()
            up, down = some[1].bool() & ~nan, some[2].bool() & ~nan
            assert bool(torch.isnan(got[nan]).all()), "NaN by right"
            assert bool((got[up] == float("inf")).all()) and bool((got[down] == -float("inf")).all()), "infinite by right"
            fin = ~(nan | up | down)
            err = (got - o[cq[b]:cq[b + 1], h]).abs()
            assert bool((err <= tol[cq[b]:cq[b + 1], h])[fin].all()), "finite"
    assert fd.fd_device_status(clear=True) == fd.FD_OK


# ------------------------------------------------------------------ the key splits' plan
def planned(lens, keys, hq, hkv, known=True):
    """Split count that fd_prompt plans: its workspace's size over one split's."""
    q = torch.empty(sum(lens), hq, D, dtype=torch.float16, device=DEV)
    k = torch.empty(sum(keys), hkv, D, dtype=torch.float16, device=DEV)
    kw = dict(batch=len(lens), max_q=max(lens) if known else 0, max_k=max(keys) if known else 0)
    size = fd.fd_prompt_workspace_size(fd.make_prompt_desc(q, k, k, **kw))
    return size // (q.shape[0] * hq * 130 * 4) if size else 1


def test_prompt_plan_counts_every_sequence():
    """Each sequence has a query tile of its own: many short ones fill the SMs, and
    cutting their keys only adds parts."""
    assert planned([2] * 64, [9000] + [300] * 63, 32, 8) == 1
    assert planned([1] * 100, [12000] + [200] * 99, 8, 8) == 1
    assert planned([1] * 64, [9000] * 64, 16, 2) == 1
    # without max_k the keys of all sequences together are no sequence's
    assert planned([1] * 64, [300] * 64, 8, 2, known=False) == 1
    assert planned([1] * 16, [2500] * 16, 8, 8, known=False) == 1
    # one request, or a few, with long keys
    assert planned([64], [9000], 8, 2) > 8 and planned([64], [9000], 8, 2, known=False) > 8
    assert planned([1] * 4, [9000, 100, 100, 100], 32, 8) > 1
    assert planned([1] * 4, [9000] * 4, 32, 8) == 2


@pytest.mark.parametrize("known", [True, False])
def test_prompt_ragged_short_queries(known):
    """What the plan leaves whole and what it cuts, against the definition."""
    for lens, keys, hq, hkv in (([2] * 20, [3000] + [100] * 19, 8, 2), ([1, 3, 0, 2], [4000, 50, 10, 700], 6, 2)):
        q, k, v, cq, ck = prompt_case(41, "bf16", lens, keys, hq, hkv)
        d = fd.make_prompt_desc(q, k, v, batch=len(lens), max_k=max(keys) if known else 0)
        size = fd.fd_prompt_workspace_size(d)
        out, lse = torch.full(q.shape, NAN, device=DEV), torch.full(q.shape[:2], NAN, device=DEV)
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV) if size else None
        fd.check(fd.fd_prompt(d, q, k, v, i32(cq), i32(ck), out, lse, ws))
        o, z, tol, ltol = ref.prompt(q, k, v, cq, ck, True, torch.float32)
        ref.close(out, o, tol, "out")
        ref.close(lse, z, ltol, "lse")


# ------------------------------------------------------------------ the store's tiles
@pytest.mark.parametrize("n", [257, 1024, 1025])
def test_store_single_rows_of_many_requests(n):
    """A step of as many requests as decide the tile of the launch, some skipped."""
    held = [(k * 977) % 300 for k in range(n)]
    k, v, slots, caches, scales = store_case(n, "bf16", [1] * n, held, 2, 16, 16)
    slots[5::11] = -1
    run_store(k, v, slots, caches, scales, 16, 16)


@pytest.mark.parametrize("lens,held", [([300, 1, 90], [7, 63, 0]), ([1000], [5]), ([3] * 120, [k % 70 for k in range(120)])])
def test_store_prompt_rows_across_tiles(lens, held):
    run_store(*store_case(len(lens), "f16", lens, held, 3, 64, 32), 64, 32)


# ------------------------------------------------------------------ calls that the contracts allow
def test_prompt_special_values_of_many_sequences():
    """More sequences than are sorted: the rows to redo are found in the order of the sequences."""
    lens = [int(x) for x in np.random.default_rng(5).integers(1, 60, size=140)]
    q, k, v, cq, ck = prompt_case(51, "f16", lens, lens, 4, 2)
    for b in range(0, 140, 3):                     # behind the first query of every third sequence
        v[cq[b + 1] - 1, b % 2, b % D] = NAN
    out, _ = run_prompt(q, k, v, cq, ck, True)
    o, _, tol, _ = ref.prompt(q, k, torch.nan_to_num(v), cq, ck, True, torch.float32)
    hit = torch.zeros_like(out, dtype=torch.bool)
    for b in range(0, 140, 3):
        hit[cq[b + 1] - 1, 2 * (b % 2):2 * (b % 2) + 2, b % D] = True
    assert bool(torch.isnan(out[hit]).all())
    assert bool(((out.double() - o).abs() <= tol)[~hit].all())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1)])
def test_prompt_head_stride_of_one_head_is_never_used(hq, hkv):
    q, k, v, cq, ck = prompt_case(52, "bf16", [150], [150], hq, hkv)
    zero = lambda x: x.as_strided(x.shape, (x.stride(0), 0, 1))
    want = run_prompt(q, k, v, cq, ck, True)
    got = run_prompt(zero(q) if hq == 1 else q, zero(k), zero(v), cq, ck, True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("q_len,G", [(16, 16), (16, 2), (1, 128), (5, 13)])
def test_scaled_decode_wide_query_blocks(q_len, G):
    lens = [3, 500, 0, 1025]
    case = scaled_case(G, "bf16", lens, q_len, G, 1, 32, 16)
    check_scaled(*case, lens, 32, 16)


def test_scaled_decode_reads_scales_that_heads_and_blocks_share():
    """One K scale for all heads, one V scale for all blocks of a head: strides of 0 are the decode's to read."""
    lens = [700, 33]
    q, caches, scales, table = scaled_case(53, "f16", lens, 1, 8, 2, 16, 16)
    shared = [scales[0][:, :1].expand(-1, 2, -1), scales[1][:1].expand(scales[1].shape[0], -1, -1)]
    check_scaled(q, caches, shared, table, lens, 16, 16)


def test_prompt_captured_with_key_splits_replays_on_new_inputs():
    q, k, v, cq, ck = prompt_case(54, "bf16", [60, 5], [4000, 300], 6, 2)
    d = fd.make_prompt_desc(q, k, v, batch=2, max_k=4000)
    ws = torch.empty(fd.fd_prompt_workspace_size(d), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    out, lse, a, b = torch.zeros(q.shape, device=DEV), torch.zeros(q.shape[:2], device=DEV), i32(cq), i32(ck)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run = lambda: fd.check(fd.fd_prompt(d, q, k, v, a, b, out, lse, ws))
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        for cut in (4000, 100, 4300):              # the sequences' border moves on the GPU
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=gen(cut), device=DEV))
            b.copy_(i32([0, cut, 4300]))
            graph.replay()
            side.synchronize()
            o, z, tol, ltol = ref.prompt(q, k, v, cq, [0, cut, 4300], True, torch.float32)
            ref.close(out, o, tol, "out")
            ref.close(lse, z, ltol, "lse")


def test_calls_on_two_streams_at_once():
    """Prompts, stores and decodes of two requests' programs, each on a stream and with buffers of its own."""
    jobs = []
    for s in range(2):
        q, k, v, cq, ck = prompt_case(60 + s, "bf16", [700 + 90 * s, 33], [900, 33 + s], 8, 2)
        lens = [4000 + s, 77]
        jobs.append((torch.cuda.Stream(), (q, k, v, cq, ck), (*scaled_case(70 + s, "f16", lens, 1, 8, 2, 16, 16), lens)))
    want = [(run_prompt(*p, True), run_scaled(*c[:4], c[4], 16, 16)) for _, p, c in jobs]
    got = [[], []]

    def work(i):
        stream, p, c = jobs[i]
        torch.cuda.set_device(DEV)
        with torch.cuda.stream(stream):
            for _ in range(10):
                got[i].append((run_prompt(*p, True), run_scaled(*c[:4], c[4], 16, 16)))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 10
        for (po, pl), (so, sl) in got[i]:
            assert torch.equal(po.nan_to_num(7), want[i][0][0].nan_to_num(7)) and torch.equal(pl.nan_to_num(7), want[i][0][1].nan_to_num(7))
            assert torch.equal(so, want[i][1][0]) and torch.equal(sl, want[i][1][1])


def test_cache_offsets_past_32_bits():
    """A pool of 70000 pages, 4.6 GB each of K and V: rows stored and read at its end, as in a small pool."""
    H, page, block, far = 8, 64, 16, 70000
    pages = [far - 1, 3, far - 7, 35001]
    n = 3 * page + 9
    g = gen(80)
    k, v = randn(g, "bf16", n, H, D), randn(g, "bf16", n, H, D)
    q = randn(g, "bf16", 1, 1, 16, D)
    got = []
    for pool, where in ((far, pages), (4, [3, 0, 1, 2])):
        caches = [torch.zeros(pool, H, page, D, dtype=torch.uint8, device=DEV).view(ref.F8) for _ in range(2)]
        scales = [torch.ones(pool, H, page // block, device=DEV) for _ in range(2)]
        at = torch.tensor(where, device=DEV)
        t = torch.arange(n, device=DEV)
        slots = at[t // page] * page + t % page
        fd.check(fd.fd_cache_store(fd.make_store_desc(k, v, *caches, page_size=page), fd.make_scales(*scales, block=block),
                                   k, v, slots, *caches))
        out, lse = run_scaled(q, caches, scales, at[None].to(torch.int32), [n], page, block)
        got.append([out, lse] + [x.view(torch.uint8)[at] for x in caches] + [s[at] for s in scales])
        del caches, scales
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert float(got[0][0].abs().max()) > 0


def test_prompt_offsets_past_32_bits():
    """Rows 131072 elements apart: the last ones lie 9 GB behind the first."""
    n, last = 35000, 200
    g = gen(81)
    wide = torch.zeros(n, 1024, D, dtype=torch.bfloat16, device=DEV)
    q, k, v = wide[:, :4], wide[:, 500:502], wide[:, 1022:]
    for x in (q, k, v):
        x[-last:] = randn(g, "bf16", last, x.shape[1], D)
    small = [x[-last:].contiguous() for x in (q, k, v)]
    d = fd.make_prompt_desc(q, k, v, batch=1, max_q=last, max_k=last, n_splits=1)
    out, lse = torch.zeros(n, 4, D, device=DEV), torch.zeros(n, 4, device=DEV)
    fd.check(fd.fd_prompt(d, q, k, v, i32([n - last, n]), i32([n - last, n]), out, lse))
    want, wl = run_prompt(*small, [0, last], [0, last], True, n_splits=1)
    assert torch.equal(out[-last:], want) and torch.equal(lse[-last:], wl) and not bool(out[:-last].any())
