"""fd_qkv_rope on the GPU against 64 bits (pages_ref.rope: the tolerance of 32-bit
arithmetic is derived there; each output adds half a step of its type)."""
import math

import pytest
import torch

import pages_ref as ref
import split_kv_gb300 as fd

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D = 128
F8 = torch.float8_e4m3fn
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


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


class Step:
    def __init__(self, seed, n, hq, hkv, dtype="bf16", cache="same", page=16, norm=True, rot=128, pairs=False, wtype=None, per_head=False,
                 fused=True, far=5000, eps=1e-6, scale=1.0, theta=10000.0, weights=True, k_rows=False, pool=None, tokens_first=False):
        g = gen(seed)
        T = DT[dtype]
        self.T, self.hq, self.hkv, self.page, self.norm, self.rot, self.pairs, self.eps, self.scale = T, hq, hkv, page, norm, rot, pairs, eps, scale
        x = torch.randn(n, hq + 2 * hkv, D, generator=g, device=DEV) * 2
        x[..., 5::37] *= 8
        x = x.to(T)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        wt = T if wtype is None else wtype
        shape = lambda h: (h, D) if per_head else (D,)
        self.qw = (1 + 0.4 * torch.randn(shape(hq), generator=g, device=DEV)).to(wt) if norm and weights else None
        self.kw = (1 + 0.4 * torch.randn(shape(hkv), generator=g, device=DEV)).to(wt) if norm and weights else None
        self.freq = ref.inv_freq(theta, rot).to(DEV) if rot else None
        self.pos = torch.randint(0, far + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        self.kc = self.vc = self.slots = None
        self.ks, self.vs = 1 / 16, 3 / 64
        if cache != "none":
            kind = F8 if cache == "e4m3" else T
            if page:
                lead, tok = (-(-n // page) + 3 if pool is None else pool), page
            else:
                lead, tok = 3, n // 2 + 7
            shape = (lead, tok, hkv, D) if tokens_first else (lead, hkv, tok, D)
            self.kc, self.vc = (torch.randn(shape, generator=g, device=DEV).to(kind) for _ in range(2))
            if tokens_first:
                self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
            self.slots = torch.randperm(lead * tok, generator=g, device=DEV)[:n]
        self.q_out = torch.full((n, hq, D), 7.0, dtype=T, device=DEV)
        self.k_out = torch.full((n, hkv, D), 7.0, dtype=T, device=DEV) if cache == "none" or k_rows else None

    def desc(self):
        return fd.make_rope_desc(self.q, self.k, self.v, q_out=self.q_out, k_out=self.k_out, k_cache=self.kc, v_cache=self.vc,
                                 page_size=self.page if self.kc is not None else 0, q_weight=self.qw, k_weight=self.kw, norm_q=self.norm,
                                 norm_k=self.norm, rot_dim=self.rot, interleaved=self.pairs, eps=self.eps, rot_scale=self.scale,
                                 k_scale=self.ks, v_scale=self.vs)

    def call(self, d=None, stream=None):
        fd.check(fd.fd_qkv_rope(d or self.desc(), self.q, self.k, self.v, self.qw, self.kw, self.freq, self.pos, self.slots, self.q_out,
                                self.k_out, self.kc, self.vc, stream=stream), "fd_qkv_rope")

    def want(self):
        """(name, value, tolerance) of each output before the call's effects are read."""
        out = []
        there = self.pos >= 0
        freq = self.freq.tolist() if self.rot else []
        q, eq = ref.rope(self.q, self.qw, self.norm, self.pos, freq, self.rot, self.pairs, self.eps, self.scale)
        k, ek = ref.rope(self.k, self.kw, self.norm, self.pos, freq, self.rot, self.pairs, self.eps, self.scale)
        for name, rows, err, buf in (("q_out", q, eq, self.q_out), ("k_out", k, ek, self.k_out)):
            if buf is None:
                continue
            value, tol = buf.double(), torch.zeros(buf.shape, dtype=torch.float64, device=DEV)
            value[there], tol[there] = rows[there], err[there] + ref.rounding(rows[there], self.T)
            out.append((name, value, tol))
        if self.kc is not None:
            tok = self.kc.shape[2]
            put = there & (self.slots >= 0) & (self.slots < self.kc.shape[0] * tok)
            lead, off = self.slots[put] // tok, self.slots[put] % tok
            for name, cache, rows, err, s in (("k_cache", self.kc, k, ek, self.ks), ("v_cache", self.vc, self.v.double(), torch.zeros_like(ek), self.vs)):
                value = cache.double()
                tol = torch.zeros_like(value)
                rows, err = rows[put], err[put]
                if cache.dtype == F8:
                    # the reciprocal and the product with it round once each
                    rows, err = rows / s, err / s + 2.0 ** -23 * rows.abs() / s
                    rows = torch.where(torch.isfinite(rows), rows.clamp(-448, 448), float("nan"))
                t = err + ref.rounding(rows, cache.dtype) if name == "k_cache" or cache.dtype == F8 else torch.zeros_like(err)
                for a, v in ((value, rows), (tol, t)):
                    a.transpose(1, 2)[lead, off] = v.to(a.dtype)
                out.append((name, value, tol))
        return out

    def check(self, want):
        for name, value, tol in want:
            buf = {"q_out": self.q_out, "k_out": self.k_out, "k_cache": self.kc, "v_cache": self.vc}[name]
            ref.close(buf, value, tol, name)


def one(*a, **kw):
    s = Step(*a, **kw)
    want = s.want()
    s.call()
    torch.cuda.synchronize()
    s.check(want)
    return s


@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (1, 8, 8), (2, 5, 1), (3, 12, 4), (64, 32, 8), (65, 6, 2), (257, 64, 8), (1000, 3, 3), (5000, 32, 8)])
@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "none")])
@pytest.mark.parametrize("pairs", [False, True])
def test_rope(n, hq, hkv, dtype, cache, pairs):
    one(n + hq, n, hq, hkv, dtype, cache, pairs=pairs)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotated_part(rot, pairs, norm):
    one(rot + 1, 70, 7, 3, "f16", rot=rot, pairs=pairs, norm=norm, k_rows=True, scale=1.2)


@pytest.mark.parametrize("wtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("per_head", [False, True])
def test_weights(wtype, per_head):
    one(5, 90, 10, 5, "bf16", wtype=wtype, per_head=per_head)


@pytest.mark.parametrize("rot,pairs", [(0, False), (16, True), (48, False), (64, True), (96, False), (112, True), (128, False)])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_rotated_part_of_many_rows(rot, pairs, cache):
    """Enough rows for items of sixteen, the last of them in part."""
    one(rot + 2, 900, 21, 5, "bf16", cache, rot=rot, pairs=pairs, k_rows=True, scale=0.9)


@pytest.mark.parametrize("wtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("page", [0, 32])
def test_weights_of_many_rows(wtype, per_head, page):
    one(50, 1200, 18, 9, "f16", wtype=wtype, per_head=per_head, page=page)


@pytest.mark.parametrize("n", [40, 1500, 9000])
def test_heads_apart(n):
    """Rows whose heads do not lie end to end, and ones whose tokens share a value row (a stride of 0)."""
    s = Step(51, n, 12, 6, "bf16", "same")
    x = torch.randn(n, 24, D, generator=gen(52), device=DEV).to(s.T)
    s.q, s.k, s.v = x[:, ::2], x[:, 1:13:2], x[:1, :6].expand(n, 6, D)
    want = s.want()
    s.call()
    s.check(want)


def test_norm_without_weights_and_eps():
    one(6, 50, 4, 2, "f16", weights=False, eps=0.5)
    one(7, 50, 4, 2, "bf16", weights=False, eps=0.0)


@pytest.mark.parametrize("far", [1, 131072, 10 ** 6, 2 ** 31 - 1])
def test_far_positions(far):
    """The 64-bit reference's own angle, position * inv_freq, is off by 2^-53 of itself: 2.4e-7 at 2^31."""
    s = Step(8, 300, 4, 2, "f16", cache="none", norm=False, far=far)
    s.pos[0], s.pos[1] = far, 0
    want = s.want()
    if far > 10 ** 6:
        extra = 2.0 ** -53 * far * 2
        want = [(n, v, t + extra * v.abs().amax(-1, keepdim=True) * 2) for n, v, t in want]
    s.call()
    s.check(want)


@pytest.mark.parametrize("freq", [0.0, 1.0, -0.3, 3.75, 1e-20, 1e-38, 1e-42, 7.25e3])
def test_frequencies(freq):
    s = Step(9, 200, 2, 1, "f16", cache="none", norm=False, far=3000, rot=32)
    s.freq = torch.full((16,), freq, dtype=torch.float32, device=DEV)
    want = s.want()
    s.call()
    s.check(want)


@pytest.mark.parametrize("page,tokens_first", [(0, False), (8, False), (64, True), (128, False)])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_cache_layouts(page, tokens_first, cache):
    one(10 + page, 150, 6, 3, "bf16", cache, page=page, tokens_first=tokens_first, fused=False)


def test_left_out_rows_and_slots():
    s = Step(11, 100, 4, 2, "bf16", k_rows=True)
    s.pos[[0, 50, 99]] = -1
    s.pos[51] = -2 ** 31
    s.slots[[1, 50, 98]] = -1
    s.slots[2] = -2 ** 63
    s.slots[0] = 1 << 60            # of a row that is left out: nothing to report
    want = s.want()
    s.call()
    s.check(want)
    assert fd.fd_device_status(clear=True) == fd.FD_OK
    s.slots[3], s.slots[4] = s.kc.shape[0] * 16, 2 ** 62
    s.call()
    assert fd.fd_device_status(clear=True) == fd.FD_ERR_DEVICE_BOUNDS


def test_in_place():
    for dtype in ("f16", "bf16"):
        a, b = (Step(12, 333, 9, 4, dtype, "none") for _ in range(2))
        a.call()
        b.q_out, b.k_out = b.q, b.k
        v = b.v.clone()
        b.call()
        assert torch.equal(a.q_out, b.q) and torch.equal(a.k_out, b.k) and torch.equal(v, b.v)


def test_only_queries_or_keys():
    s = Step(13, 77, 6, 2, "bf16", "same", k_rows=True)
    s.call()
    q2, kc2, vc2 = torch.zeros_like(s.q_out), s.kc.clone(), s.vc.clone()
    k2 = torch.zeros_like(s.k_out)
    d = fd.make_rope_desc(s.q, None, q_out=q2, q_weight=s.qw)
    fd.check(fd.fd_qkv_rope(d, s.q, None, None, s.qw, None, s.freq, s.pos, None, q2, None, None, None))
    d = fd.make_rope_desc(None, s.k, s.v, k_out=k2, k_weight=s.kw, k_cache=kc2, v_cache=vc2, page_size=16, k_scale=1.0)
    fd.check(fd.fd_qkv_rope(d, None, s.k, s.v, None, s.kw, s.freq, s.pos, s.slots, None, k2, kc2, vc2))
    assert torch.equal(q2, s.q_out) and torch.equal(k2, s.k_out) and torch.equal(kc2, s.kc) and torch.equal(vc2, s.vc)


def test_values_that_are_not_finite():
    """An infinity or NaN stays in its row (with the norm) or its pair (without); E4M3 stores NaN."""
    for cache in ("same", "e4m3"):
        s = Step(14, 40, 4, 4, "bf16", cache, norm=False, rot=64)
        s.q[3, 1, 100] = float("inf")
        s.k[4, 2, 90] = float("-inf")
        s.k[5, 0, 127] = float("nan")
        s.v[6, 3, 0], s.v[6, 3, 1], s.v[7, 0, 5] = float("inf"), float("-inf"), float("nan")
        s.v[8, 0, :] = 3e4
        want = s.want()
        s.call()
        if cache == "same":         # infinities as they are
            assert s.q_out[3, 1, 100] == float("inf")
        for name, value, tol in want:
            buf = {"q_out": s.q_out, "k_cache": s.kc, "v_cache": s.vc}[name]
            fin = torch.isfinite(value)
            assert torch.equal(torch.isfinite(buf.float()), fin) and torch.equal(torch.isnan(buf.float()), torch.isnan(value))
            ref.close(torch.where(fin, buf.double(), 0.0), torch.where(fin, value, 0.0), tol.nan_to_num(0, 0, 0), name)
    s = Step(15, 20, 4, 2, "f16", "none")
    s.q[2, 1, 3] = float("nan")
    s.call()
    nan = torch.isnan(s.q_out)
    assert bool(nan[2, 1].all()) and int(nan.sum()) == D


def test_rows_of_zeros_and_large_values():
    s = Step(16, 30, 3, 2, "bf16", "same", eps=1e-6)
    s.q[0], s.k[1] = 0, 0
    s.q[2], s.k[2] = 1e17, -1e17
    s.q[3] = 1e-18
    want = s.want()
    s.call()
    s.check(want)
    assert not bool(s.q_out[0].any())


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements, and slots behind them."""
    page, hkv = 64, 8
    pool = (1 << 32) // (page * hkv * D) + 40
    s = Step(17, 200, 4, hkv, "bf16", "none")
    s.k_out = None
    s.page = page
    s.ks = s.vs = 0.25
    s.kc, s.vc = (torch.zeros(pool, hkv, page, D, dtype=F8, device=DEV) for _ in range(2))
    s.slots = torch.arange(200, device=DEV) * 7 + (pool - 30) * page
    k, _ = ref.rope(s.k, s.kw, True, s.pos, s.freq.tolist(), 128, False, s.eps, 1.0)
    s.call()
    lead, off = s.slots // page, s.slots % page
    got = s.kc.view(torch.uint8)[lead, :, off].view(F8).double() * s.ks
    assert float((got - k).abs().max() / k.abs().max()) < 2.0 ** -4
    got = s.vc.view(torch.uint8)[lead, :, off].view(F8).double() * s.vs
    assert float((got - s.v.double()).abs().max() / s.v.double().abs().max()) < 2.0 ** -4
    assert int((s.kc.view(torch.uint8)[:pool - 40] != 0).sum()) == 0


def test_stream_and_graph():
    s = Step(18, 500, 8, 4, "bf16", "same")
    d = s.desc()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = s.want()
    s.call(d, stream=side)
    side.synchronize()
    s.check(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call(d)
    for k in range(3):
        o = Step(30 + k, 500, 8, 4, "bf16", "same", far=10 ** (k + 2))
        s.q.copy_(o.q), s.k.copy_(o.k), s.v.copy_(o.v), s.pos.copy_(o.pos), s.slots.copy_(o.slots)
        want = s.want()
        graph.replay()
        torch.cuda.synchronize()
        s.check(want)


def test_same_bits_whatever_the_batch():
    """A token's result does not depend on what else is in the call."""
    s = Step(19, 3000, 8, 2, "bf16", "none")
    s.call()
    for a, b in ((0, 1), (17, 90), (2990, 3000)):
        q, k = torch.zeros(b - a, 8, D, dtype=s.T, device=DEV), torch.zeros(b - a, 2, D, dtype=s.T, device=DEV)
        d = fd.make_rope_desc(s.q[a:b], s.k[a:b], q_out=q, k_out=k, q_weight=s.qw, k_weight=s.kw)
        fd.check(fd.fd_qkv_rope(d, s.q[a:b], s.k[a:b], None, s.qw, s.kw, s.freq, s.pos[a:b].contiguous(), None, q, k, None, None))
        assert torch.equal(q, s.q_out[a:b]) and torch.equal(k, s.k_out[a:b])


@pytest.mark.parametrize("n", [40, 900])
@pytest.mark.parametrize("scale", [1 / 64, 2.0 ** -126])
def test_e4m3_of_large_finite_values(n, scale):
    """A finite value whose quotient by the scale overflows 32 bits is beyond 448 like any other: 448, not NaN.
    Infinities and NaN stay NaN."""
    s = Step(21, n, 4, 4, "bf16", "e4m3", norm=False, rot=64)
    s.ks = s.vs = scale
    s.v[6, 3, :4] = torch.tensor([1e37, -3.3e38, float("inf"), float("nan")], device=DEV)
    s.k[7, 2, 64:68] = torch.tensor([3.3e38, -1e37, float("-inf"), float("nan")], device=DEV)   # (of the part that is not rotated)
    s.k[8, 1, 3], s.pos[8] = 1e37, 3                                                           # of a rotated pair
    s.call()
    tok = s.kc.shape[2]
    rows = lambda cache, t, h: cache[s.slots[t] // tok, h, s.slots[t] % tok].float()
    v, k, turned = rows(s.vc, 6, 3)[:4], rows(s.kc, 7, 2)[64:68], rows(s.kc, 8, 1)
    assert v[:2].tolist() == [448.0, -448.0] and bool(torch.isnan(v[2:]).all())
    assert k[:2].tolist() == [448.0, -448.0] and bool(torch.isnan(k[2:]).all())
    a = 3 * float(s.freq[3])
    want = [math.copysign(448.0, math.cos(a)), math.copysign(448.0, math.sin(a))]
    assert [float(turned[3]), float(turned[3 + 32])] == want
    assert int(torch.isnan(s.kc.float()).sum()) == 2 and int(torch.isnan(s.vc.float()).sum()) == 2


@pytest.mark.parametrize("pairs", [False, True])
def test_rows_beyond_32_bit_offsets(pairs):
    """Queries and keys, in and out, of more than 2^31 elements each."""
    n, h = (1 << 31) // (16 * D) + 1500, 16
    s = Step(23, 1, h, h, "bf16", "none", pairs=pairs)
    block = (torch.randn(5000, h, D, generator=gen(24), device=DEV) * 2).to(s.T)
    x = block.repeat(-(-n // 5000), 1, 1)[:n]
    pos = torch.randint(0, 100000, (n,), generator=gen(25), device=DEV, dtype=torch.int32)
    q_out, k_out = torch.zeros_like(x), torch.zeros_like(x)
    d = fd.make_rope_desc(x, x, q_out=q_out, k_out=k_out, q_weight=s.qw, k_weight=s.kw, interleaved=pairs)
    fd.check(fd.fd_qkv_rope(d, x, x, None, s.qw, s.kw, s.freq, pos, None, q_out, k_out, None, None))
    for a, b in ((0, 300), (n // 2 - 100, n // 2 + 100), (n - 1700, n)):
        for got, w in ((q_out, s.qw), (k_out, s.kw)):
            want, err = ref.rope(x[a:b], w, True, pos[a:b], s.freq.tolist(), 128, pairs, s.eps, 1.0)
            ref.close(got[a:b], want, err + ref.rounding(want, s.T), (a, b))
