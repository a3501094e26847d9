"""A serving loop over a paged cache, operator after operator as a program calls them:
page tables, heads' norms and rotation into the cache, decode, forks with their
copies, rejected drafts, a compaction.  The decode is compared with plain 64-bit
attention over keys rotated in 64 bits; what only moves pages must not change
a bit of it."""
import math

import pytest
import torch

import pages_ref as ref
import split_kv_gb300 as fd

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from split_kv_gb300 import _build
    _build.build()
    torch.cuda.set_device(DEV)
    fd.fd_device_status(clear=True)
    yield


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    """One layer, `rows` sequences, a pool of pages; every call as in a loop that never reads the GPU."""

    def __init__(self, kind, rows=12, page=16, width=40, pool=200, hq=8, hkv=2, seed=1):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        self.kind, self.rows, self.page, self.pool, self.hq, self.hkv = kind, rows, page, pool, hq, hkv
        self.T = torch.bfloat16
        self.table = torch.zeros(rows, width, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(pool, generator=self.g, device=DEV).to(torch.int32)
        self.count, self.shares = i32([pool]), torch.zeros(pool, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
        dtype = F8 if kind == "e4m3" else self.T
        # what nobody has written yet is NaN in a 16-bit cache
        self.kc, self.vc = (torch.full((pool, hkv, page, D), float("nan"), device=DEV).to(dtype) for _ in range(2))
        self.ks, self.vs = (1 / 8, 1 / 16) if kind == "e4m3" else (1.0, 1.0)
        self.kw, self.qw = ((1 + 0.2 * torch.randn(D, generator=self.g, device=DEV)).to(self.T) for _ in range(2))
        self.freq = ref.inv_freq(10000.0, D).to(DEV)
        self.src, self.dst, self.n = i32([-1] * pool), i32([-1] * pool), i32([0])
        self.pages = fd.make_page_desc(self.table, self.free, None, copies=self.src, page_size=page, n_pages=pool)
        self.pools = fd.make_pools([self.kc, self.vc])
        self.said = [[] for _ in range(rows)]           # the oracle's rows (k rotated in 64 bits, v) of each sequence

    def append(self, new):
        """New tokens for each sequence, through tables, norms, rotation and the cache."""
        n = sum(new)
        slots = torch.full((n + 3,), 7, dtype=torch.int64, device=DEV)
        pos = torch.full((n + 3,), 7, dtype=torch.int32, device=DEV)
        d = fd.make_page_desc(self.table, self.free, slots, page_size=self.page, n_pages=self.pool)
        held = self.lens.tolist()
        fd.check(fd.fd_page_tables(d, self.lens, i32(new), self.free, self.count, self.table, self.lens, self.count, None, slots, pos))
        x = (torch.randn(n + 3, self.hq + 2 * self.hkv, D, generator=self.g, device=DEV) * 2).to(self.T)
        q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]
        q_out = torch.zeros(n + 3, self.hq, D, dtype=self.T, device=DEV)
        rd = fd.make_rope_desc(q, k, v, q_out=q_out, k_cache=self.kc, v_cache=self.vc, page_size=self.page, q_weight=self.qw,
                               k_weight=self.kw, k_scale=self.ks, v_scale=self.vs)
        fd.check(fd.fd_qkv_rope(rd, q, k, v, self.qw, self.kw, self.freq, pos, slots, q_out, None, self.kc, self.vc))
        at = 0
        for b, m in enumerate(new):
            p = torch.arange(held[b], held[b] + m, device=DEV)
            y, _ = ref.rope(k[at:at + m], self.kw, True, p, self.freq.tolist(), D, False, 1e-6, 1.0)
            self.said[b] += list(zip(y, v[at:at + m].double()))
            at += m

    def decode(self):
        g = torch.Generator(device=DEV)
        g.manual_seed(99)
        q = torch.randn(self.rows, self.hq, D, generator=g, device=DEV).to(self.T)
        out, lse = torch.zeros(self.rows, self.hq, D, device=DEV), torch.zeros(self.rows, self.hq, device=DEV)
        d = fd.make_desc(q, self.kc, self.vc, page_size=self.page, max_pages_per_seq=self.table.shape[1], max_seqlen=640, n_splits=3,
                         k_scale=self.ks, v_scale=self.vs)
        ws = torch.empty(fd.fd_workspace_size(d, 3), dtype=torch.uint8, device=DEV)
        fd.check(fd.fd_decode(d, q, self.kc, self.vc, self.lens, self.table, out, lse, ws))
        return q, out, lse

    def check(self):
        """The decode against 64 bits: keys and values carry one rounding to the cache's type each (of the
        key, half a step relative of each element: |dot| moves by at most u sum |q k|), the rest
        is decode's own 32-bit arithmetic."""
        q, out, lse = self.decode()
        u = torch.finfo(self.kc.dtype).eps / 2
        tiny = 2.0 ** -10 * max(self.ks, self.vs) if self.kind == "e4m3" else 2.0 ** -133
        for b, rows in enumerate(self.said):
            assert int(self.lens[b]) == len(rows)
            if not rows:
                assert not bool(out[b].any()) and bool((lse[b] == -math.inf).all())
                continue
            k, v = torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
            for h in range(self.hq):
                kk, vv, qq = k[:, h * self.hkv // self.hq], v[:, h * self.hkv // self.hq], q[b, h].double()
                s = kk @ qq / math.sqrt(D)
                w = torch.softmax(s, 0)
                ds = (u * kk.abs() + tiny + 2.0 ** -18 * kk.abs()) @ qq.abs() / math.sqrt(D) + 2.0 ** -14
                e = 2 * float(ds.max()) * math.exp(2 * float(ds.max()))
                tol = (w * 1.0) @ (vv.abs() * (e + u) + tiny) + 2.0 ** -12
                got, want = out[b, h].double(), w @ vv
                assert bool(((got - want).abs() <= tol).all()), (b, h, float((got - want).abs().max()), float(tol.min()))
                assert abs(float(lse[b, h]) - float(torch.logsumexp(s, 0))) <= float(ds.max()) + 1e-3

    def copies(self):
        fd.check(fd.fd_page_copy(self.pools, self.src, self.dst, self.n))

    def fork(self, parents, children, keep):
        fd.check(fd.fd_page_fork(self.pages, i32(parents), i32(children), i32(keep), self.lens, self.free, self.count, self.table, self.shares,
                                 self.lens, self.count, self.src, self.dst, self.n))
        self.copies()
        for p, c, k in zip(parents, children, keep):
            self.said[c] = self.said[p][:k]

    def trim(self, keep):
        fd.check(fd.fd_page_trim(self.pages, i32(keep), self.lens, self.free, self.count, self.table, self.shares, self.lens, self.count,
                                 self.src, self.dst, self.n))
        self.copies()
        self.said = [s if k < 0 or k >= len(s) else s[:k] for s, k in zip(self.said, keep)]

    def compact(self, n_keep):
        fd.check(fd.fd_page_compact(self.pages, n_keep, self.lens, self.free, self.count, self.table, self.shares, self.count, self.src,
                                    self.dst, self.n))
        self.copies()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_serving_loop(kind):
    s = Server(kind)
    s.append([100, 37, 0, 16, 1, 0, 0, 0, 0, 0, 0, 250])
    s.check()
    s.append([1, 1, 0, 1, 1, 0, 0, 0, 0, 0, 0, 1])
    s.check()
    # samples of two prompts, one cut back; each goes its own way
    s.fork([0, 0, 11, 11, 11], [5, 6, 7, 8, 9], [101, 101, 251, 250, 48])
    s.check()
    s.append([1, 0, 0, 0, 0, 3, 4, 1, 20, 1, 0, 1])
    s.check()
    # drafts that are not taken: decode as before them, bit by bit
    before = s.decode()[1:]
    lens, free, count = s.lens.tolist(), s.free.tolist(), int(s.count)
    s.append([4, 4, 0, 4, 4, 4, 4, 4, 4, 4, 0, 4])
    s.trim(lens)
    after = s.decode()[1:]
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert int(s.count) == count and s.free.tolist()[:count] == free[:count]
    # some end, some are cut back into what they share
    s.trim([60, 0, -1, 10, -1, 50, 101, 100, -1, 48, -1, 0])
    s.check()
    s.append([30, 5, 0, 9, 0, 20, 1, 40, 2, 3, 8, 0])
    s.check()
    # tight: the upper part of the pool is given up, and nothing changes
    before = s.decode()[1:]
    used = s.pool - int(s.count)
    s.compact(used + 5)
    after = s.decode()[1:]
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert int(s.count) == 5 and int(s.table[:, :].max()) >= 0
    live = {int(p) for b in range(s.rows) for p in s.table[b, :-(-len(s.said[b]) // s.page)]}
    assert len(live) == used and max(live) < used + 5
    for page in range(used + 5, s.pool):              # and could be overwritten
        s.kc.view(torch.uint8)[page] = 0x7f
    s.check()
    s.trim([0] * s.rows)
    assert int(s.count) == used + 5 and not bool(s.shares.any()) and sorted(s.free.tolist()[:used + 5]) == list(range(used + 5))
    assert fd.fd_device_status(clear=True) == fd.FD_OK
