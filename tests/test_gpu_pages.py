"""fd_page_fork, fd_page_trim, fd_page_compact and fd_page_copy on the GPU: whole
numbers and bytes, so equal to the plain implementations of pages_ref.py."""
import numpy as np
import pytest
import torch

import pages_ref as ref
import split_kv_gb300 as fd

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class State:
    """Lengths, tables, sharing counts and the free stack of a pool, as lists."""

    def __init__(self, seed, batch, page, width, held=0.6, spare=40, longest=None, empty=0):
        r = self.r = np.random.default_rng(seed)
        self.page, self.width = page, width
        longest = page * width if longest is None else longest
        self.lens = [int(x) for x in r.integers(0, longest + 1, size=batch)]
        for b in range(batch):
            if r.random() < 0.2:
                self.lens[b] = self.lens[b] // page * page
            if r.random() >= held or b >= batch - empty:
                self.lens[b] = 0
        have = [-(-x // page) for x in self.lens]
        self.n_pages = sum(have) + spare
        perm = [int(x) for x in r.permutation(self.n_pages)]
        self.table, at = [], 0
        for h in have:
            self.table.append(perm[at:at + h] + [-9] * (width - h))
            at += h
        self.free = perm[at:]
        self.count = len(self.free)
        self.free += [-5] * (self.n_pages - self.count + 3)
        self.shares = [0] * self.n_pages

    def take(self, out):
        self.lens, self.count, self.table, self.free = out["lens"], out["count"], out["table"], out["free"]
        self.shares = out["shares"] if out["shares"] is not None else self.shares

    def forked(self, n):
        """n forks of random parts into sequences that hold nothing."""
        empty = [b for b, x in enumerate(self.lens) if x == 0]
        full = [b for b, x in enumerate(self.lens) if x > 0]
        n = min(n, len(empty))
        if not full or n == 0:
            return [], [], []
        children = [int(x) for x in self.r.permutation(empty)[:n]]
        parents = [int(self.r.choice(full)) for _ in range(n)]
        keep = [int(self.r.integers(0, self.lens[p] + 1)) if self.r.random() < 0.6 else self.lens[p] for p in parents]
        return parents, children, keep


def device(s, alias, n_lists, shared=True):
    t = dict(lens=i32(s.lens), count=i32([s.count]), table=i32(s.table).view(len(s.lens), s.width), free=i32(s.free),
             shares=i32(s.shares) if shared else None, src=i32([77] * n_lists), dst=i32([78] * n_lists), n=i32([79]))
    t["lens_out"], t["count_out"] = (t["lens"], t["count"]) if alias else (torch.full_like(t["lens"], 99), torch.full_like(t["count"], 99))
    t["desc"] = fd.make_page_desc(t["table"], t["free"], None, copies=t["src"], page_size=s.page, n_pages=s.n_pages)
    return t


def run_fork(s, parents, children, keep, alias=False, stream=None):
    t = device(s, alias, max(1, len(parents)))
    args = (t["desc"], i32(parents), i32(children), None if keep is None else i32(keep), t["lens"], t["free"], t["count"], t["table"],
            t["shares"], t["lens_out"], t["count_out"], t["src"], t["dst"], t["n"])
    fd.check(fd.fd_page_fork(*args), "fd_page_fork")
    torch.cuda.synchronize()
    return t


def run_trim(s, keep, alias=False, shared=True):
    t = device(s, alias, len(s.lens) if shared else 0, shared)
    lists = (t["src"], t["dst"], t["n"]) if shared else (None, None, t["n"])
    fd.check(fd.fd_page_trim(t["desc"], i32(keep), t["lens"], t["free"], t["count"], t["table"], t["shares"], t["lens_out"],
                             t["count_out"], *lists), "fd_page_trim")
    torch.cuda.synchronize()
    return t


def run_compact(s, n_keep, n_lists, alias=False, shared=True):
    t = device(s, alias, n_lists, shared)
    fd.check(fd.fd_page_compact(t["desc"], n_keep, t["lens"], t["free"], t["count"], t["table"], t["shares"], t["count_out"], t["src"],
                                t["dst"], t["n"]), "fd_page_compact")
    torch.cuda.synchronize()
    t["lens_out"] = t["lens"]
    return t


def same(t, want, bad=False):
    for name, a in (("count", t["count_out"]), ("n", t["n"])):
        assert int(a) == want[name], name
    for name in ("table", "free", "shares", "src", "dst"):
        if want.get(name) is not None and t[name] is not None:
            assert t[name].tolist() == want[name], name
    if "lens" in want:
        assert t["lens_out"].tolist() == want["lens"]
    assert fd.fd_device_status(clear=True) == (fd.FD_ERR_DEVICE_BOUNDS if bad else fd.FD_OK)


def want_fork(s, parents, children, keep):
    n = max(1, len(parents))
    return ref.fork(parents, children, keep, s.lens, s.free, s.count, s.table, s.shares, s.page, s.n_pages, [77] * n, [78] * n)


def want_trim(s, keep, shared=True):
    n = len(s.lens) if shared else 0
    return ref.trim(keep, s.lens, s.free, s.count, s.table, s.shares if shared else None, s.page, s.n_pages, [77] * n, [78] * n)


def want_compact(s, n_keep, n, shared=True):
    return ref.compact(n_keep, s.lens, s.free, s.count, s.table, s.shares if shared else None, s.page, s.n_pages, [77] * n, [78] * n)


SIZES = [(2, 16, 5, 1), (9, 8, 40, 4), (40, 16, 130, 25), (300, 32, 12, 200), (64, 16, 1100, 60), (3000, 16, 3, 1500), (8192, 8, 2, 5000)]


# ------------------------------------------------------------------ forks
@pytest.mark.parametrize("batch,page,width,n", SIZES)
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("whole", [False, True])
def test_fork(batch, page, width, n, alias, whole):
    s = State(batch + page, batch, page, width, held=0.45, spare=n + 20, empty=1)
    parents, children, keep = s.forked(n)
    keep = None if whole else keep
    want, bad = want_fork(s, parents, children, keep)
    assert not bad
    same(run_fork(s, parents, children, keep, alias), want)


def test_fork_many_of_one_parent():
    for tokens in (16 * 700, 16 * 700 + 5):
        s = State(3, 200, 16, 701, held=0.0, spare=900)
        s.table[4] = s.free[:701]
        s.free = s.free[701:900] + [-5] * 30
        s.lens[4], s.count = tokens, 199
        children = [b for b in range(200) if b != 4]
        keep = [tokens if b % 5 else tokens - 16 * (b % 3) for b in children]
        for k in (None, keep):
            want, bad = want_fork(s, [4] * 199, children, k)
            assert not bad
            same(run_fork(s, [4] * 199, children, k), want)


@pytest.mark.parametrize("what", ["few pages", "no pages", "child twice", "child holds tokens", "itself", "too long", "negative", "outside",
                                  "bad length", "free count", "bad free page", "bad table entry", "child of a child"])
def test_fork_reports_what_does_not_fit(what):
    s = State(5, 12, 16, 30, held=1.0, spare=30, empty=6)
    parents, children, keep = [0, 1, 2, 3, 1], [6, 7, 8, 9, 10], [20, 35, 17, 33, 40]
    s.lens[:4], s.n_pages = [200, 100, 90, 50], 100
    perm = [int(x) for x in s.r.permutation(100)]
    s.table = [perm[7 * b:7 * b + 7] * 2 + [-9] * 16 for b in range(12)]
    s.free, s.count, s.shares = perm[84:] + [-5] * 9, 16, [0] * 100
    s.lens[4:] = [0] * 8
    s.lens[11] = 3
    if what == "few pages":
        s.count = 3
    elif what == "no pages":
        s.count = 0
    elif what == "child twice":
        children[3] = 7
    elif what == "child holds tokens":
        children[2] = 11
    elif what == "itself":
        children[2] = 2
    elif what == "too long":
        keep[1] = 101
    elif what == "negative":
        keep[1] = -1
    elif what == "outside":
        parents[0], children[1], parents[2], children[3] = 12, -1, -1, 12
    elif what == "bad length":
        s.lens[1] = 16 * 30 + 1
    elif what == "free count":
        s.count = len(s.free) + 4
    elif what == "bad free page":
        s.free[14] = 100
    elif what == "bad table entry":
        s.table[0][0] = 100
        s.table[1][1] = -1
    elif what == "child of a child":          # (nothing to report: parents as they were, without tokens)
        parents[3], keep[3] = 6, 0
    want, bad = want_fork(s, parents, children, keep)
    assert bad == (what != "child of a child")
    same(run_fork(s, parents, children, keep), want, bad)


def test_fork_of_nothing():
    s = State(6, 5, 16, 4)
    want, bad = want_fork(s, [], [], [])
    t = device(s, False, 1)
    fd.check(fd.fd_page_fork(t["desc"], None, None, None, t["lens"], t["free"], t["count"], t["table"], t["shares"], t["lens_out"],
                             t["count_out"], t["src"], t["dst"], t["n"], n_forks=0))
    same(t, want, bad)


# ------------------------------------------------------------------ trims
def shared_state(seed, batch, page, width, n):
    """A state after forks and some trims, so that pages are shared in all ways."""
    s = State(seed, batch, page, width, held=0.5, spare=2 * n + batch + 20)
    for _ in range(2):
        parents, children, keep = s.forked(n)
        out, bad = want_fork(s, parents, children, keep)
        assert not bad
        s.take(out)
    return s


def random_keep(s, r):
    keep = []
    for x in s.lens:
        u = r.random()
        keep.append(0 if u < 0.2 else x if u < 0.3 else -1 if u < 0.35 else int(r.integers(0, x + 1)) if u < 0.7 else max(0, x - int(r.integers(0, 6))) if u < 0.9
                    else x // s.page * s.page // 2)
    return keep


@pytest.mark.parametrize("batch,page,width,n", SIZES)
@pytest.mark.parametrize("alias", [False, True])
def test_trim(batch, page, width, n, alias):
    s = shared_state(batch + 7 * page, batch, page, width, n)
    for _ in range(3):
        keep = random_keep(s, s.r)
        want, bad = want_trim(s, keep)
        assert not bad
        same(run_trim(s, keep, alias), want)
        s.take(want)
    want, bad = want_trim(s, [0] * batch)              # and everything goes back
    same(run_trim(s, [0] * batch, alias), want)
    assert want["count"] == s.n_pages and not any(want["shares"]) and sorted(want["free"][:s.n_pages]) == list(range(s.n_pages))


@pytest.mark.parametrize("batch,width", [(64, 500), (64, 2600)])
def test_trim_of_more_than_a_threads_registers_hold(batch, width):
    s = State(batch + width, batch, 16, width, held=1.0, spare=batch * 3 + 20)
    s.lens[batch - 1] = 0
    for keep in ([0] * batch, [x // 7 for x in s.lens]):
        want, bad = want_trim(s, keep, False)
        assert not bad
        same(run_trim(s, keep, shared=False), want)
    # half of the sequences become forks of a long one
    long = max(range(batch), key=lambda b: s.lens[b])
    children = [b for b in range(1, batch, 2) if b != long]
    for b in children:
        s.lens[b], s.table[b] = 0, [-9] * width
    out, bad = want_fork(s, [long] * len(children), children, [s.lens[long] - (b * 31) % 200 for b in children])
    assert not bad
    s.take(out)
    keep = [x if b % 3 else x // 5 for b, x in enumerate(s.lens)]
    want, bad = want_trim(s, keep)
    assert not bad
    same(run_trim(s, keep), want)


@pytest.mark.parametrize("count", [0, 1, 3, 30])
def test_trim_over_counts_that_are_too_low(count):
    """Eight sequences that end inside one page of which shares knows nothing: reported, within bounds."""
    s = State(3, 8, 16, 6, held=1.0, spare=40)
    s.lens = [40] * 8
    s.table = [[1, 2, 3, -9, -9, -9] for _ in range(8)]
    s.n_pages, s.shares = 40, [0] * 40
    s.free, s.count = list(range(4, 40)) + [-5] * 4, count
    t = run_trim(s, [20] * 8)
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS
    assert 0 <= int(t["count_out"]) <= 40 and 0 <= int(t["n"]) <= count
    assert all(0 <= x < 40 for row in t["table"].tolist() for x in row[:3]) and t["lens_out"].tolist() == [20] * 8


@pytest.mark.parametrize("batch,page,width,n", SIZES)
def test_trim_without_shares(batch, page, width, n):
    s = State(batch * 3 + page, batch, page, width)
    keep = random_keep(s, s.r)
    want, bad = want_trim(s, keep, False)
    assert not bad
    same(run_trim(s, keep, shared=False), want)


def test_trim_undoes_a_step():
    s = State(31, 50, 16, 40, held=1.0, spare=900, longest=300)
    new = [int(x) for x in s.r.integers(0, 200, size=50)]
    t = device(s, False, 50)
    slots = torch.zeros(sum(new), dtype=torch.int64, device=DEV)
    d = fd.make_page_desc(t["table"], t["free"], slots, page_size=16, n_pages=s.n_pages)
    fd.check(fd.fd_page_tables(d, t["lens"], i32(new), t["free"], t["count"], t["table"], t["lens_out"], t["count_out"], None, slots, None))
    fd.check(fd.fd_page_trim(t["desc"], t["lens"], t["lens_out"], t["free"], t["count_out"], t["table"], t["shares"], t["lens_out"],
                             t["count_out"], t["src"], t["dst"], t["n"]))
    assert t["lens_out"].tolist() == s.lens and int(t["count_out"]) == s.count and t["free"].tolist() == s.free


@pytest.mark.parametrize("what", ["few pages", "no pages", "bad length", "negative length", "bad page", "bad tail", "let go twice", "no room",
                                  "free count", "bad free page"])
def test_trim_reports_what_does_not_fit(what):
    s = State(9, 8, 16, 20, held=1.0, spare=30, empty=4)
    s.lens = [200, 100, 90, 50, 0, 0, 0, 0]
    s.n_pages, s.shares = 80, [0] * 80
    perm = [int(x) for x in s.r.permutation(80)]
    s.table = [perm[13 * b:13 * b + 13] + [-9] * 7 for b in range(4)] + [[-9] * 20 for _ in range(4)]
    s.free, s.count = perm[52:] + [-5] * 52, 28
    out, bad = want_fork(s, [0, 0, 1, 1], [4, 5, 6, 7], [190, 200, 100, 33])
    assert not bad
    s.take(out)
    keep = [70, 50, 10, 0, 71, 64, 40, 20]
    if what == "few pages":
        s.count = 2
    elif what == "no pages":
        s.count = 0
    elif what == "bad length":
        s.lens[1] = 16 * 20 + 1
    elif what == "negative length":
        s.lens[2] = -4
    elif what == "bad page":
        s.table[3][1] = 80
        s.table[0][9] = -1
    elif what == "bad tail":
        s.table[0][4] = 80
    elif what == "let go twice":
        s.table[3][0] = s.table[2][5]
        s.shares[s.table[2][5]] = 0
    elif what == "no room":
        s.free = s.free[:s.count + 3]
    elif what == "free count":
        s.count = -1
    elif what == "bad free page":
        s.free[s.count - 1] = 80
    want, bad = want_trim(s, keep)
    assert bad
    same(run_trim(s, keep), want, True)


def test_trim_of_no_sequences():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    table, free = torch.empty(0, 4, dtype=torch.int32, device=DEV), i32([3, 2, 1])
    d = fd.make_page_desc(table, free, None, page_size=16, n_pages=4)
    out = i32([-1])
    fd.check(fd.fd_page_trim(d, e, e, free, i32([2]), table, None, e, out))
    assert int(out) == 2 and free.tolist() == [3, 2, 1]


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("batch,page,width,n", SIZES)
@pytest.mark.parametrize("part", [0.0, 0.3, 0.8, 1.0])
def test_compact(batch, page, width, n, part):
    s = shared_state(batch + 11 * page, batch, page, width, n)
    keep = random_keep(s, s.r)
    s.take(want_trim(s, keep)[0])
    n_keep = int(s.n_pages * part)
    want, bad = want_compact(s, n_keep, s.n_pages)
    same(run_compact(s, n_keep, s.n_pages, alias=batch % 2 == 0), want, bad)
    few = max(0, want["n"] - 2)
    want, bad = want_compact(s, n_keep, few)                  # a copy list that is too short
    same(run_compact(s, n_keep, few), want, bad)
    want, bad = want_compact(s, n_keep, s.n_pages, False)
    same(run_compact(s, n_keep, s.n_pages, shared=False), want, bad)


def test_compact_a_large_pool():
    """More free pages than one round of the filter holds, and more than one word of the map a thread."""
    s = State(17, 40, 8, 300, held=0.9, spare=400000)
    for n_keep in (1000, 200000, 399000):
        want, bad = want_compact(s, n_keep, s.n_pages)
        assert bad == (n_keep == 1000)
        same(run_compact(s, n_keep, s.n_pages), want, bad)


def test_compact_as_large_as_it_gets():
    """8192 sequences, and as many pages behind n_keep as a call takes."""
    s = State(29, 8192, 8, 2, held=0.5, spare=fd.FD_MAX_COMPACT_PAGES)
    n_keep = s.n_pages - fd.FD_MAX_COMPACT_PAGES
    want, bad = want_compact(s, n_keep, 20000)
    assert not bad and want["n"] > 1000
    same(run_compact(s, n_keep, 20000), want)


def test_forks_as_many_as_a_call_takes():
    s = State(31, 8192, 8, 3, held=0.4, spare=9000)
    children = [b for b, x in enumerate(s.lens) if x == 0]
    parents = [int(x) for x in s.r.integers(0, 8192, size=8192)]
    children = (children * 3)[:8192]                     # (most of them twice)
    want, bad = want_fork(s, parents, children, None)
    assert bad and want["n"] > 100
    same(run_fork(s, parents, children, None), want, True)


def test_compact_of_many_segments():
    s = State(23, 200, 16, 1100, held=1.0, spare=30000)
    for n_keep in (s.n_pages - s.count + 5000, s.n_pages - s.count):
        want, bad = want_compact(s, n_keep, s.n_pages)
        assert not bad and want["n"] > 10000
        same(run_compact(s, n_keep, s.n_pages), want)


@pytest.mark.parametrize("what", ["bad length", "bad page", "bad free page", "free count"])
def test_compact_reports(what):
    s = State(19, 6, 16, 20, held=1.0, spare=50)
    s.lens[2], s.lens[3] = max(s.lens[2], 40), max(s.lens[3], 40)
    if what == "bad length":
        s.lens[2] = 16 * 20 + 1
    elif what == "bad page":
        s.table[3][1], s.table[3][0] = s.n_pages, -1
    elif what == "bad free page":
        s.free[3], s.free[4] = -1, s.n_pages
    else:
        s.count = len(s.free) + 1
    want, bad = want_compact(s, s.n_pages // 2, s.n_pages)
    assert bad
    same(run_compact(s, s.n_pages // 2, s.n_pages), want, True)


# ------------------------------------------------------------------ copies
def copied(x, pairs):
    y = x.clone()
    for a, b in pairs:
        if a >= 0 and b >= 0:
            y[b] = x[a]
    return y


def rand_bytes(seed, dtype, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    return torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV, generator=g).view(dtype).view(shape)


def bits(x):
    return x.contiguous().view(torch.uint8)


POOLS = {
    "bf16": lambda P: [rand_bytes(k, torch.bfloat16, P, 8, 16, 128) for k in range(5)],
    "many": lambda P: [rand_bytes(k, torch.float16, P, 2, 8, 128) for k in range(70)],
    "tokens first": lambda P: [rand_bytes(1, torch.float16, P, 16, 4, 128).permute(0, 2, 1, 3)],
    "heads apart": lambda P: [rand_bytes(2, torch.float16, 3, P, 16, 128).permute(1, 0, 2, 3)],
    "part of rows": lambda P: [rand_bytes(3, torch.bfloat16, P, 2, 16, 2, 128)[:, :, :, k] for k in range(2)],
    "e4m3 and scales": lambda P: [rand_bytes(4, torch.float8_e4m3fn, P, 8, 64, 128)] + [rand_bytes(5 + k, torch.float32, P, 8, 2) for k in range(3)],
    "odd": lambda P: [rand_bytes(6, torch.uint8, P, 5, 7), rand_bytes(7, torch.int16, P, 3, 5), rand_bytes(8, torch.float32, P, 7),
                      rand_bytes(9, torch.float64, P, 3), rand_bytes(10, torch.uint8, P)],
    "offset": lambda P: [rand_bytes(11, torch.float32, P * 40 + 1)[1:].view(P, 2, 20), rand_bytes(12, torch.bfloat16, P * 64 + 3)[3:].view(P, 64)],
    "large": lambda P: [rand_bytes(13, torch.float16, P, 16, 128, 128)],
    "steps": lambda P: [rand_bytes(14, torch.float32, P, 6)[:, ::2]],
}


@pytest.mark.parametrize("name", sorted(POOLS))
@pytest.mark.parametrize("pairs", [1, 7, 11])
def test_copy(name, pairs):
    P = 23
    pools = POOLS[name](P)
    perm = [int(x) for x in np.random.default_rng(pairs).permutation(P)]
    src, dst = perm[:pairs], perm[pairs:2 * pairs]
    if pairs > 1:
        src[1] = src[0]                       # one page into two
        src[2], dst[3] = -1, -1               # left out
        dst[4] = src[4]
    want = [copied(x, zip(src, dst)) for x in pools]
    fd.check(fd.fd_page_copy(fd.make_pools(pools), i32(src), i32(dst)))
    for x, y in zip(pools, want):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("count", [0, 3, 9, 20, -2])
def test_copy_counts(count):
    P = 40
    x = rand_bytes(1, torch.float16, P, 4, 16, 128)
    src, dst = list(range(9)), list(range(20, 29))
    want = copied(x, list(zip(src, dst))[:max(0, count)])
    fd.check(fd.fd_page_copy(fd.make_pools([x]), i32(src), i32(dst), i32([count])))
    assert torch.equal(bits(x), bits(want))


def test_copy_reports_pages_outside_the_pool():
    x = rand_bytes(2, torch.float16, 10, 4, 16, 128)
    want = copied(x, [(1, 2)])
    fd.check(fd.fd_page_copy(fd.make_pools([x]), i32([10, 1, 3]), i32([4, 2, 1 << 30])))
    assert torch.equal(bits(x), bits(want))
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS


def test_copy_writes_nothing_else():
    """The bytes between the rows of strided pools, and behind the last page, stay."""
    back = rand_bytes(3, torch.float16, 9, 4, 20, 160)
    x = back[:, :, :16, :128]
    before = back.clone()
    fd.check(fd.fd_page_copy(fd.make_pools([x]), i32([1, 2]), i32([8, 0])))
    want = before.clone()
    want[8, :, :16, :128], want[0, :, :16, :128] = before[1, :, :16, :128], before[2, :, :16, :128]
    assert torch.equal(bits(back), bits(want))


# ------------------------------------------------------------------ streams and graphs
def test_page_operators_captured():
    """Fork, copy, trim and compaction in one graph, replayed over other lengths in the same buffers."""
    s = State(41, 20, 16, 30, held=1.0, spare=200, empty=8)
    cache = rand_bytes(5, torch.float16, s.n_pages, 2, 16, 128)
    start = cache.clone()
    t = device(s, False, s.n_pages)
    fork = device(s, False, 8)
    lens2, count2, count3 = (torch.zeros_like(x) for x in (t["lens"], t["count"], t["count"]))
    parents, children, keep = i32([0] * 8), i32(list(range(12, 20))), i32([0] * 8)
    cut = i32([-1] * 20)
    pools = fd.make_pools([cache])

    def step():
        fd.check(fd.fd_page_fork(fork["desc"], parents, children, keep, t["lens"], t["free"], t["count"], t["table"], t["shares"],
                                 t["lens_out"], t["count_out"], fork["src"], fork["dst"], fork["n"]))
        fd.check(fd.fd_page_copy(pools, fork["src"], fork["dst"], fork["n"]))
        fd.check(fd.fd_page_trim(t["desc"], cut, t["lens_out"], t["free"], t["count_out"], t["table"], t["shares"], lens2, count2,
                                 t["src"], t["dst"], t["n"]))
        fd.check(fd.fd_page_copy(pools, t["src"], t["dst"], t["n"]))
        fd.check(fd.fd_page_compact(t["desc"], s.n_pages * 3 // 4, lens2, t["free"], count2, t["table"], t["shares"], count3, t["src"],
                                    t["dst"], t["n"]))
        fd.check(fd.fd_page_copy(pools, t["src"], t["dst"], t["n"]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                      # (attributes are set once per context, ahead of the capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    fd.fd_device_status(clear=True)
    for seed in range(3):
        n = State(50 + seed, 20, 16, 30, held=1.0, spare=200, empty=8)
        n.n_pages = s.n_pages
        perm = [int(x) for x in n.r.permutation(s.n_pages)]
        n.lens = [min(x, 300) for x in n.lens]
        have = [-(-x // 16) for x in n.lens]
        while sum(have) + 60 > s.n_pages * 3 // 4:
            n.lens = [x // 2 for x in n.lens]
            have = [-(-x // 16) for x in n.lens]
        at = np.concatenate([[0], np.cumsum(have)])
        n.table = [perm[at[b]:at[b + 1]] + [-9] * (30 - have[b]) for b in range(20)]
        n.free = perm[at[-1]:]
        n.count = len(n.free)
        n.free += [-5] * (len(s.free) - n.count)
        n.shares = [0] * s.n_pages
        par, chi, kp = n.forked(8)
        kt = [int(n.r.integers(-1, x + 1)) for x in n.lens[:12]] + [int(n.r.integers(0, k + 1)) for _, k in sorted(zip(chi, kp))]
        for dst, v in ((t["lens"], n.lens), (t["count"], [n.count]), (t["table"], n.table), (t["free"], n.free), (t["shares"], n.shares),
                       (parents, par), (children, chi), (keep, kp), (cut, kt)):
            dst.copy_(i32(v).view(dst.shape))
        cache.copy_(start)
        want = start.clone()
        # the tokens that each sequence stands for, followed through the reference
        out, bad = want_fork(n, par, chi, kp)
        assert not bad
        want = copied(want, zip(out["src"][:out["n"]], out["dst"][:out["n"]]))
        n.take(out)
        out, bad = ref.trim(kt, n.lens, n.free, n.count, n.table, n.shares, 16, n.n_pages, [77] * n.n_pages, [78] * n.n_pages)
        assert not bad
        want = copied(want, zip(out["src"][:out["n"]], out["dst"][:out["n"]]))
        n.take(out)
        out, bad = want_compact(n, n.n_pages * 3 // 4, n.n_pages)
        assert not bad
        want = copied(want, zip(out["src"][:out["n"]], out["dst"][:out["n"]]))
        graph.replay()
        torch.cuda.synchronize()
        assert t["table"].tolist() == out["table"] and t["shares"].tolist() == out["shares"] and int(count3) == out["count"]
        assert lens2.tolist() == n.lens and t["free"].tolist() == out["free"] and int(t["n"]) == out["n"]
        assert torch.equal(bits(cache), bits(want))


def test_copies_of_several_shapes_captured():
    """Launches of one call that overlap each other still come behind what wrote the list and the pages,
    and before what reads them."""
    P = 300
    pools = [rand_bytes(20, torch.bfloat16, P, 8, 16, 128), rand_bytes(21, torch.float32, P, 8, 2), rand_bytes(22, torch.bfloat16, P, 2, 8, 128),
             rand_bytes(23, torch.uint8, P, 5, 3)]
    first = [x.clone() for x in pools]
    src, dst, n = i32([0] * 100), i32([0] * 100), i32([0])
    given = [i32([0] * 100), i32([0] * 100), i32([0])]
    handle = fd.make_pools(pools)
    after = [torch.empty_like(x) for x in pools]

    def step():
        for x, y in zip(pools, first):
            bits(x).copy_(bits(y))
        for x, y in zip((src, dst, n), given):
            x.copy_(y)
        fd.check(fd.fd_page_copy(handle, src, dst, n))
        for x, y in zip(after, pools):
            bits(x).copy_(bits(y))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(5):
        perm = [int(x) for x in np.random.default_rng(seed).permutation(P)]
        m = 100 - seed * 20
        for x, v in zip(given, (perm[:100], perm[100:200], [m])):
            x.copy_(i32(v))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(after, first):
            assert torch.equal(bits(x), bits(copied(y, list(zip(perm[:100], perm[100:200]))[:m])))


def test_two_streams_at_once():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    s = [shared_state(70 + k, 300, 16, 40, 100) for k in range(2)]
    keep = [random_keep(x, x.r) for x in s]
    want = [want_trim(x, k)[0] for x, k in zip(s, keep)]
    t = [device(x, False, 300) for x in s]
    cut = [i32(k) for k in keep]
    torch.cuda.synchronize()
    for x, k, st in zip(t, cut, (a, b)):
        fd.check(fd.fd_page_trim(x["desc"], k, x["lens"], x["free"], x["count"], x["table"], x["shares"], x["lens_out"], x["count_out"],
                                 x["src"], x["dst"], x["n"], stream=st))
    torch.cuda.synchronize()
    for x, w in zip(t, want):
        same(x, w)


# ------------------------------------------------------------------ copies of several shapes, behind what writes their list
def mixed_pools(P, layers, seed=200):
    """Keys, values and the scales of both, layer after layer, with a pool of odd rows here and there."""
    out = []
    for k in range(layers):
        out += [rand_bytes(seed + 5 * k, torch.float8_e4m3fn, P, 4, 32, 128), rand_bytes(seed + 5 * k + 1, torch.float8_e4m3fn, P, 4, 32, 128),
                rand_bytes(seed + 5 * k + 2, torch.float32, P, 4, 2), rand_bytes(seed + 5 * k + 3, torch.float32, P, 4, 2)]
        if k % 5 == 0:
            out.append(rand_bytes(seed + 5 * k + 4, torch.uint8, P, 3, 7))
    return out


@pytest.mark.parametrize("layers", [1, 6, 36])
def test_copy_of_pools_in_any_order(layers):
    """One launch takes the pools of a shape wherever they are in the list (36 layers: more than a launch takes)."""
    P = 20
    pools = mixed_pools(P, layers)
    perm = [int(x) for x in np.random.default_rng(layers).permutation(P)]
    src, dst = perm[:9], perm[9:18]
    src[3], dst[5] = -1, -1
    want = [copied(x, zip(src, dst)) for x in pools]
    fd.check(fd.fd_page_copy(fd.make_pools(pools), i32(src), i32(dst)))
    for x, y in zip(pools, want):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("captured", [False, True])
def test_copies_of_several_shapes_behind_forks_and_trims(captured):
    """Lists that a fork and a trim write directly ahead of the copies, over and over: every launch of a
    copy sees the list of the call before it, not that of the repetition before, and its pages."""
    states = []
    for seed in range(2):
        s = State(90 + seed, 40, 16, 12, held=0.6, spare=200, empty=12)
        s.n_pages = 480
        perm = [int(x) for x in s.r.permutation(480)]
        have = [-(-x // 16) for x in s.lens]
        at = np.concatenate([[0], np.cumsum(have)])
        s.table = [perm[at[b]:at[b + 1]] + [-9] * (12 - have[b]) for b in range(40)]
        s.free = perm[at[-1]:]
        s.count = len(s.free)
        s.free += [-5] * (480 - s.count)
        s.shares = [0] * 480
        parents, children, keep = s.forked(8)
        start = dict(lens=s.lens, count=[s.count], table=s.table, free=s.free, shares=s.shares, parents=parents, children=children, keep=keep)
        forked, bad = want_fork(s, parents, children, keep)
        assert not bad and forked["n"] > 2
        s.take(forked)
        cut = random_keep(s, s.r)
        trimmed, bad = want_trim(s, cut)
        assert not bad and trimmed["n"] > 0
        pairs = [list(zip(o["src"], o["dst"]))[:o["n"]] for o in (forked, trimmed)]
        states.append(({k: i32(v) for k, v in dict(start, cut=cut).items()}, pairs, trimmed))
    pools = mixed_pools(480, 3)
    first = [x.clone() for x in pools]
    want = []
    for _, pairs, _ in states:
        y = first
        for p in pairs:
            y = [copied(x, p) for x in y]
        want.append(y)
    handle = fd.make_pools(pools)
    now = {k: v.clone() for k, v in states[0][0].items()}
    given = {k: v.clone() for k, v in now.items()}
    table = now["table"].view(40, 12)
    src, dst, n, lens2, count2 = i32([-1] * 40), i32([-1] * 40), i32([0]), torch.zeros_like(now["lens"]), i32([0])
    desc = fd.make_page_desc(table, now["free"], None, copies=src, page_size=16, n_pages=480)

    def step():
        for x, y in zip(pools, first):
            bits(x).copy_(bits(y))
        for k in now:
            now[k].copy_(given[k])
        src.fill_(-1), dst.fill_(-1), n.zero_()
        fd.check(fd.fd_page_fork(desc, now["parents"], now["children"], now["keep"], now["lens"], now["free"], now["count"], table,
                                 now["shares"], lens2, count2, src, dst, n))
        fd.check(fd.fd_page_copy(handle, src, dst, n))
        fd.check(fd.fd_page_trim(desc, now["cut"], lens2, now["free"], count2, table, now["shares"], lens2, count2, src, dst, n))
        fd.check(fd.fd_page_copy(handle, src, dst, n))

    step()
    torch.cuda.synchronize()
    run = step
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for k in range(60):
        values, _, out = states[k % 2]
        for name in given:
            given[name].copy_(values[name])
        run()
        for x, y in zip(pools, want[k % 2]):
            wrong += (bits(x) != bits(y)).sum()
        wrong += (lens2 != i32(out["lens"])).sum() + (table != i32(out["table"])).sum()
    assert int(wrong) == 0
    assert fd.fd_device_status(clear=True) == fd.FD_OK


# ------------------------------------------------------------------ long rows: stages in turn, last pieces, rows apart
LONG = {    # pools, their tensors' shape behind the pages, the part that the k-th pool is, rows of a page, pieces of a row
    "pages of 32 KB": (64, (8, 32, 128), lambda k, x: x, 1, 2),
    "16400": (40, (16400,), lambda k, x: x, 1, 2),                                          # a last piece of 16 bytes
    "40976, apart": (12, (3, 41024), lambda k, x: x[:, :, :40976], 3, 3),                   # one of 8208, 48 bytes between the rows
    "8208, apart in two dimensions": (6, (4, 6, 8256), lambda k, x: x[:, :3, :5, :8208] if k % 2 else x.permute(0, 2, 1, 3)[:, :5, :3, :8208], 15, 1),
    "8192, heads ahead of pages": (14, (5, 8192), lambda k, x: x.view(5, -1, 8192).permute(1, 0, 2), 5, 1),
}


@pytest.mark.parametrize("name", sorted(LONG))
def test_copy_of_long_rows(name):
    """Thirteen pieces and more for each of the CTAs (two an SM), so that every stage is used again and again;
    pairs are left out among them, and what lies between the rows stays."""
    n, shape, part, rows, pieces = LONG[name]
    P, pairs = 190, 90
    back = [rand_bytes(300 + k, torch.uint8, P, *shape) for k in range(n)]
    before = [x.clone() for x in back]
    perm = [int(x) for x in np.random.default_rng(n).permutation(P)]
    src, dst = perm[:pairs], perm[pairs:2 * pairs]
    for k in range(0, pairs, 7):
        src[k] = src[1]
    for k in range(3, pairs, 11):
        dst[k] = -1
    dst[50] = src[50]
    counted = [(a, b) for a, b in zip(src, dst) if b >= 0 and a != b][:pairs]
    assert len(counted) * n * rows * pieces >= 13 * 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pools = fd.make_pools([part(k, x) for k, x in enumerate(back)])
    fd.check(fd.fd_page_copy(pools, i32(src), i32(dst)))
    for k, (x, y) in enumerate(zip(back, before)):
        old, new = part(k, y).clone(), part(k, y)
        for a, b in counted:
            new[b] = old[a]
        assert torch.equal(x, y), k
    fd.check(fd.fd_page_copy(pools, i32(dst), i32([-1] * 40 + src[40:]), i32([40])))        # a count that ends ahead of what counts
    for x, y in zip(back, before):
        assert torch.equal(x, y)


@pytest.mark.parametrize("row", [32768, 4096, 72])
def test_copy_beyond_32_bit_offsets(row):
    """Pages behind 2^31 and 2^32 bytes of a pool, by bulk copies and by registers."""
    P = (1 << 32) // row + 1000
    x = torch.zeros(P, row, dtype=torch.uint8, device=DEV)
    places = [3, (1 << 31) // row - 1, (1 << 31) // row + 5, (1 << 32) // row - 1, (1 << 32) // row + 7, P - 1, P - 2, 11]
    for k, q in enumerate(places):
        x[q] = rand_bytes(400 + k, torch.uint8, row)
    rows = [x[q].clone() for q in places]
    to = [P - 3, 5, P - 500, (1 << 31) // row + 9, 7, (1 << 32) // row + 2, (1 << 31) // row - 7, (1 << 32) // row - 9]
    fd.check(fd.fd_page_copy(fd.make_pools([x]), i32(places), i32(to)))
    for k in range(len(to)):
        assert torch.equal(x[to[k]], rows[k]) and torch.equal(x[places[k]], rows[k])
        x[to[k]] = 0
        x[places[k]] = 0
    assert int(x.view(-1).view(torch.int64).count_nonzero()) == 0       # (and nothing else was written)


# ------------------------------------------------------------------ trims that lack pages; large calls in a graph
@pytest.mark.parametrize("batch,width", [(600, 5), (3000, 12), (8192, 4)])
@pytest.mark.parametrize("count", [0, 9, 80])
def test_trim_that_lacks_pages_of_more_sequences_than_threads(batch, width, count):
    """More claims than free pages, numbered over several rounds of a CTA's threads."""
    s = shared_state(batch + count, batch, 16, width, batch // 3)
    keep = random_keep(s, s.r)
    claims = sum(1 for b, k in enumerate(keep) if 0 <= k < s.lens[b] and k % 16)
    s.count = min(s.count, count)
    want, bad = want_trim(s, keep)
    assert claims > s.count and bad
    same(run_trim(s, keep), want, True)


def test_large_trims_and_compactions_captured():
    """Sixteen CTAs each (more table entries than eight take), one graph over other lengths and tables."""
    batch, page, width, n_pages = 400, 16, 120, 30000
    states = []
    for seed in range(3):
        s = State(500 + seed, batch, page, width, held=0.6, spare=0)
        perm = [int(x) for x in s.r.permutation(n_pages)]
        have = [-(-x // page) for x in s.lens]
        at = np.concatenate([[0], np.cumsum(have)])
        assert at[-1] < n_pages - 2000
        s.n_pages, s.shares = n_pages, [0] * n_pages
        s.table = [perm[at[b]:at[b + 1]] + [-9] * (width - have[b]) for b in range(batch)]
        s.free = perm[at[-1]:]
        s.count = len(s.free)
        s.free += [-5] * (n_pages - s.count)
        out, bad = want_fork(s, *s.forked(100))
        assert not bad
        s.take(out)
        keep = random_keep(s, s.r)
        given = dict(lens=s.lens, count=[s.count], table=s.table, free=s.free, shares=s.shares, cut=keep)
        trimmed, bad = ref.trim(keep, s.lens, s.free, s.count, s.table, s.shares, page, n_pages, [77] * n_pages, [78] * n_pages)
        assert not bad
        s.take(trimmed)
        n_keep = n_pages // 2
        packed, bad = ref.compact(n_keep, s.lens, s.free, s.count, s.table, s.shares, page, n_pages, trimmed["src"], trimmed["dst"])
        assert not bad and packed["n"] > 1000
        states.append(({k: i32(v) for k, v in given.items()}, trimmed, packed))
    now = {k: v.clone() for k, v in states[0][0].items()}
    table = now["table"].view(batch, width)
    src, dst = i32([77] * n_pages), i32([78] * n_pages)
    n1, n2, lens2, count2, count3 = i32([0]), i32([0]), torch.zeros_like(now["lens"]), i32([0]), i32([0])
    desc = fd.make_page_desc(table, now["free"], None, copies=src, page_size=page, n_pages=n_pages)

    def step():
        fd.check(fd.fd_page_trim(desc, now["cut"], now["lens"], now["free"], now["count"], table, now["shares"], lens2, count2, src, dst, n1))
        fd.check(fd.fd_page_compact(desc, n_pages // 2, lens2, now["free"], count2, table, now["shares"], count3, src, dst, n2))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for given, trimmed, packed in states * 2:
        for k, v in given.items():
            now[k].copy_(v)
        src.fill_(77), dst.fill_(78)
        graph.replay()
        torch.cuda.synchronize()
        assert lens2.tolist() == trimmed["lens"] and int(count2) == trimmed["count"] and int(n1) == trimmed["n"]
        assert table.tolist() == packed["table"] and now["shares"].tolist() == packed["shares"] and now["free"].tolist() == packed["free"]
        assert int(count3) == packed["count"] and int(n2) == packed["n"]
        assert src.tolist() == packed["src"] and dst.tolist() == packed["dst"]
    assert fd.fd_device_status(clear=True) == fd.FD_OK


@pytest.mark.parametrize("part,lists", [(0.3, None), (0.8, 5), (0.9, 5), (0.9, None)])
def test_compact_and_the_high_end_kept_after_all(part, lists):
    """The stack as it was, from n_keep on, and the pages that moved are what is free of the high end: with
    them no page is lost, whether the compaction could finish or not."""
    s = shared_state(71, 60, 16, 30, 20)
    n_keep = int(s.n_pages * part)
    n_lists = s.n_pages if lists is None else lists
    held = {p for b, x in enumerate(s.lens) for p in s.table[b][:-(-x // 16)]}
    fits = len(held) <= n_keep and n_lists >= s.n_pages - n_keep
    kept = [p for p in s.free[:s.count] if p >= n_keep]
    want, bad = want_compact(s, n_keep, n_lists)
    assert bad == (not fits)
    t = run_compact(s, n_keep, n_lists)
    same(t, want, bad)
    table, n = t["table"].tolist(), int(t["n"])
    held = {p for b, x in enumerate(s.lens) for p in table[b][:-(-x // 16)]}
    free = t["free"].tolist()[:int(t["count_out"])] + kept + t["src"].tolist()[:n]
    assert len(free) == len(set(free)) and not held & set(free) and held | set(free) == set(range(s.n_pages))
