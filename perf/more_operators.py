"""Cases and plain forms of the operators between a model's projections and its paged cache.

Five operators that a serving loop runs around page tables, attention and decode:
  rope     norms of queries and keys for each head, rotation by position, and the new K/V rows' way into the cache
  fork     sequences that share the pages of another one's tokens
  trim     tokens taken back from the ends of sequences (rejected drafts, finished requests), their pages freed
  compact  pages moved to the low end of the pool, so that its high end can be given up
  copy     the contents of pages moved in the caches of every layer

`run` computes them with elementary torch operations, or, where `own` is set, through split_kv_gb300.
The page operators change tables, sharing counts and the free stack in place, so a pass begins by putting
back what they change (one copy, in both forms).
"""
import math

import torch

own = False
D = 128
F8 = torch.float8_e4m3fn
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _text(v):
    return ",".join(str(x) for x in v)


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the prefill step of one long prompt of a 32 / 8-head model with norms, out of one projection's output
        dict(name="rope_prefill", op="rope", lens="16384", held="0", hq=32, hkv=8, dtype="bf16", cache="same", page=16, norm=True, rot=128,
             style="half", fused=True, theta=500000.0, pad=0),
        # ragged requests, some behind a prefix, half of each head rotated; the keys also as rows, for a store with block scales
        dict(name="rope_packed", op="rope", lens="3001,17,1024,640,1,2050,333,129", held="0,12000,0,0,131000,100,0,31", hq=64, hkv=8,
             dtype="f16", cache="rows", page=64, norm=False, rot=64, style="pairs", fused=False, theta=10000.0, pad=13),
        # one new token of each of 64 running requests, into an E4M3 cache with one scale per tensor
        dict(name="rope_step", op="rope", lens=_text([1] * 64), held=_text((k * 1237) % 8000 for k in range(64)), hq=32, hkv=8, dtype="bf16",
             cache="e4m3", page=16, norm=True, rot=128, style="half", fused=True, theta=1000000.0, pad=0),
        # one token of one request of a small model without grouped heads, contiguous cache
        dict(name="rope_one", op="rope", lens="1", held="900", hq=8, hkv=8, dtype="f16", cache="same", page=0, norm=True, rot=128,
             style="half", fused=False, theta=10000.0, pad=0),
        # 64 samples of one long prompt
        dict(name="fork_samples", op="fork", lens="128003", parents=_text([0] * 64), keep="", page=16),
        # four beams each of four requests, cut back to where they part
        dict(name="fork_beams", op="fork", lens="900,3333,12001,64", parents="0,0,0,1,1,1,2,2,2,3,3,3", keep="900,880,867,3333,3333,3300,12001,12001,11999,64,48,63",
             page=16),
        # drafted tokens that the model did not take, of 64 requests
        dict(name="trim_drafts", op="trim", lens=_text(40 + (k * 977) % 8000 for k in range(64)),
             keep=_text(40 + (k * 977) % 8000 - (k * 5) % 9 for k in range(64)), group=1, prefix=0, page=16),
        # a third of 300 requests done, in groups of six that share a prompt, some of the others cut back into it
        dict(name="trim_finished", op="trim", lens=_text(2500 + (k * 3571) % 7000 for k in range(300)),
             keep=_text(0 if k % 3 == 0 else (1007 if k % 7 == 0 else 100000) for k in range(300)), group=6, prefix=2000, page=16),
        # half of a large pool given up
        dict(name="compact_half", op="compact", lens=_text(300 + (k * 3571) % 7000 for k in range(256)), group=4, prefix=256, page=16, pool=131072,
             to=65536),
        # a small pool packed tight
        dict(name="compact_small", op="compact", lens=_text(16 + (k * 577) % 2000 for k in range(32)), group=1, prefix=0, page=32, pool=2048, to=1200),
        # the moves of a compaction in the bf16 caches of 32 layers
        dict(name="copy_moves", op="copy", layers=32, pool=1024, pairs=500, hkv=8, page=16, kind="bf16", block=16),
        # the tail pages of 12 forks, E4M3 caches of 16 layers with their block scales
        dict(name="copy_tails", op="copy", layers=16, pool=256, pairs=12, hkv=8, page=64, kind="e4m3", block=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rope", "fork", "trim", "compact", "copy"])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    if op == "rope":
        hq, hkv = rng.choice([(8, 8), (12, 4), (16, 2), (32, 8), (64, 8), (5, 1), (6, 2), (1, 1)])
        n = _log(rng, 1, 200)
        top = max(1, 16384 * 48 // (hq + 2 * hkv) // n)
        lens = [1] * n if rng.random() < 0.4 else [_log(rng, 1, top) for _ in range(n)]
        held = [_log(rng, 1, 20000) if rng.random() < 0.6 else 0 for _ in range(n)]
        if n < 4 and rng.random() < 0.3:
            held[0] = _log(rng, 100000, 1000000)
        while sum(held) > 1000000 + 50000 or len(held) * max(a + b for a, b in zip(held, lens)) * hkv > 8 << 20:
            held = [x // 2 for x in held]
        return dict(op=op, lens=_text(lens), held=_text(held), hq=hq, hkv=hkv, dtype=rng.choice(["f16", "bf16"]),
                    cache=rng.choice(["same", "same", "e4m3", "rows"]), page=rng.choice([0, page, page, page]), norm=rng.random() < 0.7,
                    rot=rng.choice([128, 128, 128, 64, 32, 96, 16]), style=rng.choice(["half", "half", "pairs"]), fused=rng.random() < 0.5,
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]), pad=rng.choice([0, 0, 5, 37]))
    if op == "fork":
        n = _log(rng, 1, 8)
        lens = [_log(rng, 1, 128000 // n) for _ in range(n)]
        parents = [rng.randrange(n) for _ in range(_log(rng, 1, 64))]
        keep = "" if rng.random() < 0.5 else _text(rng.choice([lens[p], _log(rng, 1, lens[p]), lens[p] // page * page]) for p in parents)
        return dict(op=op, lens=_text(lens), parents=_text(parents), keep=keep, page=max(page, 16))
    if op in ("trim", "compact"):
        n = _log(rng, 1, 300)
        lens = [_log(rng, 1, 9000) for _ in range(n)]
        group = rng.choice([1, 1, 2, 3, 8])
        prefix = _log(rng, 1, 4000) // page * page if group > 1 else 0
        page = max(page, 16)
        if op == "trim":
            few = rng.random() < 0.4
            keep = [rng.choice([100000, x - rng.randrange(8) if few else _log(rng, 1, x), 0 if not few else x]) for x in lens]
            return dict(op=op, lens=_text(lens), keep=_text(max(0, x) for x in keep), group=group, prefix=prefix, page=page)
        live = sum(_cdiv(x, page) for x in lens)  # (at most: groups share some)
        pool = max(64, int(live * rng.choice([1.02, 1.2, 2.0])))
        return dict(op=op, lens=_text(lens), group=group, prefix=prefix, page=page, pool=pool, to=max(live, int(pool * rng.uniform(0.3, 1.0))))
    hkv = rng.choice([1, 2, 4, 8])
    layers, kind = _log(rng, 1, 32), rng.choice(["bf16", "e4m3"])
    pool = max(8, min(_log(rng, 16, 1024), (1 << 30) // (layers * hkv * page * D)))
    return dict(op=op, layers=layers, pool=pool, pairs=_log(rng, 1, pool // 2 - 1), hkv=hkv, page=page, kind=kind,
                block=rng.choice([b for b in (8, 16, 32, 64, 128) if b <= page]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _rows(g, dtype, *shape):
    """Rows of a projection: unit variance, a few channels much larger, as keys have them."""
    x = torch.randn(*shape, D, generator=g, device="cuda")
    x[..., 5::37] *= 4.0
    return x.to(DT[dtype])


def prepare(case, seed):
    st = _prepare(case, _gen(seed))
    st["case"] = case
    if own:
        _handles(case, st)
    return st


def _prepare(case, g):
    if case["op"] == "rope":
        return _prepare_rope(case, g)
    if case["op"] == "copy":
        return _prepare_copy(case, g)
    return _prepare_pages(case, g)


def _prepare_rope(case, g):
    lens, held = torch.tensor(_ints(case["lens"])), torch.tensor(_ints(case["held"]))
    hq, hkv, page, pad = case["hq"], case["hkv"], case["page"], case["pad"]
    n, B = int(lens.sum()), lens.numel()
    seq = torch.repeat_interleave(torch.arange(B), lens)
    pos = held[seq] + torch.arange(n) - (torch.cumsum(lens, 0) - lens)[seq]
    if page:  # only the pages that the new tokens reach: the others hold nothing that this step looks at
        first, pages = held // page, (held + lens + page - 1) // page - held // page
        lead, tok = int(pages.sum()) + 8, page
        perm = torch.randperm(lead, generator=g, device="cuda").cpu()
        slots = perm[(torch.cumsum(pages, 0) - pages)[seq] + pos // page - first[seq]] * page + pos % page
    else:
        lead, tok = B, int((held + lens).max())
        slots = seq * tok + pos
    behind = torch.full((pad,), -1)
    qkv = _rows(g, case["dtype"], n + pad, hq + 2 * hkv)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kind = {"same": DT[case["dtype"]], "e4m3": F8, "rows": None}[case["cache"]]
    kc = vc = None
    if kind is not None:
        kc, vc = (torch.randn(lead, hkv, tok, D, generator=g, device="cuda").to(kind) for _ in range(2))
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(DT[case["dtype"]]) if case["norm"] else None for _ in range(2)]
    rot = case["rot"]
    freq = (1.0 / case["theta"] ** (torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    return dict(q=q, k=k, v=v, qw=w[0], kw=w[1], freq=freq, pos=torch.cat([pos, behind]).to(torch.int32).cuda(),
                slots=torch.cat([slots, behind]).cuda(), kc=kc, vc=vc, q_out=torch.zeros_like(q, memory_format=torch.contiguous_format),
                k_out=torch.zeros_like(k, memory_format=torch.contiguous_format) if kind is None else None, ks=1 / 32, vs=1 / 64, eps=1e-6)


def _prepare_copy(case, g):
    layers, P, hkv, page = case["layers"], case["pool"], case["hkv"], case["page"]
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    n = case["pairs"]
    src, dst = torch.full((n + 5,), -1, dtype=torch.int32, device="cuda"), torch.full((n + 5,), -1, dtype=torch.int32, device="cuda")
    src[:n], dst[:n] = perm[:n], perm[n:2 * n]
    kind = torch.bfloat16 if case["kind"] == "bf16" else F8
    cache = torch.empty(layers, 2, P, hkv, page, D, dtype=kind, device="cuda")
    cache.view(-1).view(torch.int16).random_(generator=g)
    cache.view(-1).view(torch.int16).bitwise_and_(0x3f3f)  # finite in either type
    scales = torch.rand(layers, 2, P, hkv, page // case["block"], generator=g, device="cuda") if kind == F8 else None
    return dict(cache=cache, scales=scales, src=src, dst=dst, count=_i32([n]))


def _prepare_pages(case, g):
    """Sequences in groups that share a prompt's full pages, in a shuffled pool; what the pool has left is the free stack."""
    lens, page = _ints(case["lens"]), case["page"]
    op, dev = case["op"], "cuda"
    group, prefix = case.get("group", 1), case.get("prefix", 0)
    held = torch.tensor(lens, device=dev)
    extra = len(_ints(case["parents"])) if op == "fork" else 0
    B = len(lens) + extra
    have = (held + page - 1) // page
    gid = torch.arange(len(lens), device=dev) // group
    # what a group shares: full pages of the prompt that every one of its sequences holds
    least = torch.full((int(gid[-1]) + 1,), 1 << 30, device=dev, dtype=torch.int64).scatter_reduce(0, gid, held, "amin")
    pre_g = torch.minimum(least, torch.tensor(prefix, device=dev)) // page if group > 1 else torch.zeros_like(least)
    pre = pre_g[gid]
    own_pages = have - pre
    width = int(have.max()) + 3
    j = torch.arange(width, device=dev)
    start_g = torch.cumsum(pre_g, 0) - pre_g
    start = int(pre_g.sum()) + torch.cumsum(own_pages, 0) - own_pages
    used = int(pre_g.sum()) + int(own_pages.sum())
    pool = case["pool"] if op == "compact" else used + extra + 64
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    at = torch.where(j < pre[:, None], start_g[gid][:, None] + j, start[:, None] + j - pre[:, None]).clamp_(0, pool - 1)
    live = j < have[:, None]
    # one buffer holds what the operators change: table, sharing counts, free stack
    size = B * width + 2 * pool
    now = torch.zeros(size, dtype=torch.int32, device=dev)
    table, shares, free = now[:B * width].view(B, width), now[B * width:B * width + pool], now[B * width + pool:]
    table[:len(lens)] = torch.where(live, perm[at], torch.zeros_like(perm[at]))
    shares.copy_(torch.bincount(table[:len(lens)][live].long(), minlength=pool).sub_(1).clamp_(min=0))
    left = pool - used
    free[:left] = perm[used:]
    seqlens = torch.cat([held, torch.zeros(extra, dtype=torch.int64, device=dev)]).to(torch.int32)
    lists = max(B, pool - case["to"]) if op == "compact" else B
    st = dict(now=now, start=now.clone(), table=table, shares=shares, free=free, seqlens=seqlens, count=_i32([left]), pool=pool,
              seqlens_out=torch.zeros_like(seqlens), count_out=_i32([0]), src=torch.full((lists,), -1, dtype=torch.int32, device=dev),
              dst=torch.full((lists,), -1, dtype=torch.int32, device=dev), n_copies=_i32([0]))
    if op == "fork":
        st["parents"] = _i32(_ints(case["parents"]))
        st["children"] = torch.randperm(extra, generator=g, device=dev).to(torch.int32) + len(lens)
        st["keep"] = _i32(_ints(case["keep"])) if case["keep"] else None
    if op == "trim":
        st["keep"] = _i32(_ints(case["keep"]))
    return st


def _handles(case, st):
    """What a program that serves with split_kv_gb300 keeps between calls."""
    import split_kv_gb300 as fd
    st["fd"] = fd
    op = case["op"]
    if op == "rope":
        st["desc"] = fd.make_rope_desc(st["q"], st["k"], st["v"], q_out=st["q_out"], k_out=st["k_out"], k_cache=st["kc"], v_cache=st["vc"],
                                       page_size=case["page"], q_weight=st["qw"], k_weight=st["kw"], norm_q=case["norm"], norm_k=case["norm"],
                                       rot_dim=case["rot"], interleaved=case["style"] == "pairs", eps=st["eps"], k_scale=st["ks"], v_scale=st["vs"])
    elif op == "copy":
        pools = list(st["cache"].view(-1, *st["cache"].shape[2:]))
        if st["scales"] is not None:
            pools += list(st["scales"].view(-1, *st["scales"].shape[2:]))
        st["pools"] = fd.make_pools(pools)
    else:
        st["desc"] = fd.make_page_desc(st["table"], st["free"], None, copies=st["src"], page_size=case["page"], n_pages=st["pool"])


# ------------------------------------------------------------------ one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _pages_out(st):
    return {n: st[n] for n in ("seqlens_out", "count_out", "table", "shares", "free", "src", "dst", "n_copies")}


def _run_own(st):
    fd, op = st["fd"], st["case"]["op"]
    if op == "rope":
        fd.check(fd.fd_qkv_rope(st["desc"], st["q"], st["k"], st["v"], st["qw"], st["kw"], st["freq"], st["pos"], st["slots"], st["q_out"],
                                st["k_out"], st["kc"], st["vc"]))
        return st["q_out"], st["k_out"], st["kc"], st["vc"]
    if op == "copy":
        fd.check(fd.fd_page_copy(st["pools"], st["src"], st["dst"], st["count"]))
        return st["cache"], st["scales"]
    st["now"].copy_(st["start"])
    if op == "fork":
        fd.check(fd.fd_page_fork(st["desc"], st["parents"], st["children"], st["keep"], st["seqlens"], st["free"], st["count"], st["table"],
                                 st["shares"], st["seqlens_out"], st["count_out"], st["src"], st["dst"], st["n_copies"]))
    elif op == "trim":
        fd.check(fd.fd_page_trim(st["desc"], st["keep"], st["seqlens"], st["free"], st["count"], st["table"], st["shares"], st["seqlens_out"],
                                 st["count_out"], st["src"], st["dst"], st["n_copies"]))
    else:
        fd.check(fd.fd_page_compact(st["desc"], st["case"]["to"], st["seqlens"], st["free"], st["count"], st["table"], st["shares"],
                                    st["count_out"], st["src"], st["dst"], st["n_copies"]))
        return {n: x for n, x in _pages_out(st).items() if n != "seqlens_out"}
    return _pages_out(st)


def _run_plain(st):
    return {"rope": _plain_rope, "copy": _plain_copy, "fork": _plain_fork, "trim": _plain_trim, "compact": _plain_compact}[st["case"]["op"]](st)


def _turned(x, w, st, cos, sin):
    """Norm, then rotation, of the rows x [n, heads, D] in 32 bits."""
    case = st["case"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w.float()
    r = case["rot"]
    if case["style"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)
    return y


def _put(cache, page, slots, rows, scale):
    """Rows [n, heads, D] at their slots of a cache [pages or sequences, heads, tokens, D]."""
    tok = page or cache.shape[2]
    if cache.dtype == F8:
        rows = (rows / scale).clamp(-448, 448).to(F8).view(torch.uint8)
        cache = cache.view(torch.uint8)
    cache[slots // tok, :, slots % tok] = rows.to(cache.dtype)


def _plain_rope(st):
    at = torch.nonzero(st["pos"] >= 0).squeeze(1)
    angle = st["pos"][at].double()[:, None, None] * st["freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    k = _turned(st["k"][at], st["kw"], st, cos, sin)
    st["q_out"][at] = _turned(st["q"][at], st["qw"], st, cos, sin).to(st["q_out"].dtype)
    if st["k_out"] is not None:
        st["k_out"][at] = k.to(st["k_out"].dtype)
    if st["kc"] is not None:
        page = st["case"]["page"]
        _put(st["kc"], page, st["slots"][at], k, st["ks"])
        _put(st["vc"], page, st["slots"][at], st["v"][at].float(), st["vs"])
    return st["q_out"], st["k_out"], st["kc"], st["vc"]


def _plain_copy(st):
    i = torch.arange(st["src"].numel(), device="cuda")
    take = (i < st["count"]) & (st["src"] >= 0) & (st["dst"] >= 0)
    src, dst = st["src"][take].long(), st["dst"][take].long()
    bits = st["cache"].view(torch.int16)
    bits[:, :, dst] = bits[:, :, src]
    if st["scales"] is not None:
        st["scales"][:, :, dst] = st["scales"][:, :, src]
    return st["cache"], st["scales"]


def _plain_fork(st):
    st["now"].copy_(st["start"])
    ps, table, count = st["case"]["page"], st["table"], st["count"].long()
    parents, children = st["parents"].long(), st["children"].long()
    keep = st["seqlens"][parents].long() if st["keep"] is None else st["keep"].long()
    full, tail = keep // ps, keep % ps != 0
    upto = torch.cumsum(tail, 0)
    page = st["free"][(count - upto).clamp(min=0)]
    j = torch.arange(table.shape[1], device="cuda")
    shared = j < full[:, None]
    rows = torch.where(shared, table[parents], table[children])
    st["shares"].add_(torch.bincount(rows[shared].long(), minlength=st["pool"]))
    table[children] = torch.where((j == full[:, None]) & tail[:, None], page[:, None], rows)
    n = upto[-1]
    to = (upto - 1)[tail]
    st["src"][to] = table[parents, full.clamp(max=table.shape[1] - 1)][tail]
    st["dst"][to] = page[tail]
    st["n_copies"].copy_(n)
    st["count_out"].copy_(count - n)
    st["seqlens_out"].copy_(st["seqlens"])
    st["seqlens_out"][children] = keep.to(torch.int32)
    return _pages_out(st)


def _plain_trim(st):
    st["now"].copy_(st["start"])
    ps, table, shares, free = st["case"]["page"], st["table"], st["shares"], st["free"]
    held, keep, count = st["seqlens"].long(), st["keep"].long(), st["count"].long()
    P, (B, W) = st["pool"], table.shape
    have, stay = (held + ps - 1) // ps, (keep + ps - 1) // ps
    cut = (keep >= 0) & (keep < held)
    tail_at = (keep // ps).clamp(max=W - 1)
    tail = table.gather(1, tail_at[:, None]).squeeze(1).long()
    part = cut & (keep % ps != 0)
    may = part & (shares[tail] > 0)
    cut = cut & ~(may & (torch.cumsum(may, 0) > count))  # left as they are: no page for them
    part = part & cut
    j = torch.arange(W, device="cuda")
    gone = (cut[:, None] & (j >= stay[:, None]) & (j < have[:, None])).view(-1)
    ids = table.view(-1).long()
    left = shares - torch.bincount(ids[gone], minlength=P) - torch.bincount(tail[part], minlength=P)
    # of the sequences that keep a part of a page that no other one holds, the last keeps it, the others get copies
    b = torch.arange(B, device="cuda")
    last = torch.full((P,), -1, device="cuda").scatter_reduce(0, tail, torch.where(part, b, -1), "amax")
    moves = part & ((left[tail] >= 0) | (last[tail] != b))
    # a page that nobody holds is given back at its last place
    e = torch.arange(B * W, device="cuda")
    place = torch.full((P,), -1, device="cuda").scatter_reduce(0, ids, torch.where(gone, e, -1), "amax")
    back = gone & (left[ids] < 0) & (last[ids] < 0) & (place[ids] == e)
    upto = torch.cumsum(moves, 0)
    page = free[(count - upto).clamp(min=0)]
    base, pushed = count - upto[-1], back.sum()
    src = tail[moves].to(torch.int32)
    dst = page[moves]
    free[(base + pushed - torch.cumsum(back, 0))[back]] = ids[back].to(torch.int32)
    shares.copy_(left.clamp_(min=0))
    table.scatter_(1, tail_at[:, None], torch.where(moves, page, tail.to(torch.int32))[:, None])
    st["src"][(upto - 1)[moves]] = src
    st["dst"][(upto - 1)[moves]] = dst
    st["n_copies"].copy_(upto[-1])
    st["count_out"].copy_(base + pushed)
    st["seqlens_out"].copy_(torch.where(cut, keep, held))
    return _pages_out(st)


def _plain_compact(st):
    st["now"].copy_(st["start"])
    ps, to, table, shares, free = st["case"]["page"], st["case"]["to"], st["table"], st["shares"], st["free"]
    live = torch.arange(table.shape[1], device="cuda") < ((st["seqlens"] + ps - 1) // ps)[:, None]
    high = torch.zeros(st["pool"], dtype=torch.bool, device="cuda")
    high[table[live].long()] = True
    high[:to] = False
    movers = torch.nonzero(high).squeeze(1)
    stack = free[(torch.arange(free.numel(), device="cuda") < st["count"]) & (free < to)]
    m = min(movers.numel(), stack.numel(), st["src"].numel())
    movers, dst = movers[:m], stack.flip(0)[:m]
    names = torch.arange(st["pool"], dtype=torch.int32, device="cuda")
    names[movers] = dst
    table.copy_(torch.where(live, names[table.long()], table))
    shares[dst.long()] = shares[movers]
    shares[movers] = 0
    free[:stack.numel()] = stack
    st["src"][:m] = movers.to(torch.int32)
    st["dst"][:m] = dst
    st["n_copies"].fill_(m)
    st["count_out"].fill_(stack.numel() - m)
    return {n: x for n, x in _pages_out(st).items() if n != "seqlens_out"}


# ------------------------------------------------------------------ what a pass cannot do without
def _shared_pages(case):
    """Full pages that the groups of the case's sequences share, for each group, and its size."""
    lens, group, page = _ints(case["lens"]), case.get("group", 1), case["page"]
    if group == 1:
        return [(0, 1)] * len(lens)
    return [(min([case["prefix"]] + lens[a:a + group]) // page, len(lens[a:a + group])) for a in range(0, len(lens), group)]


def work(case):
    op, page = case["op"], case.get("page", 0)
    if op == "rope":
        n, hq, hkv = sum(_ints(case["lens"])), case["hq"], case["hkv"]
        out = {"same": 2 * 2 * D * hkv, "e4m3": 2 * D * hkv, "rows": 2 * D * hkv}[case["cache"]]
        read = hq + hkv + (0 if case["cache"] == "rows" else hkv)
        return dict(bytes=n * (2 * D * read + 2 * D * hq + out + 4 + (0 if case["cache"] == "rows" else 8)) + 2 * case["rot"],
                    flops=n * (hq + hkv) * D * ((4 if case["norm"] else 0) + 3))
    if op == "copy":
        rows = case["layers"] * 2 * case["pairs"] * case["hkv"]
        each = page * D * (2 if case["kind"] == "bf16" else 1) + (4 * (page // case["block"]) if case["kind"] == "e4m3" else 0)
        return dict(bytes=2 * rows * each + 8 * case["pairs"], flops=0)
    lens = _ints(case["lens"])
    if op == "fork":
        parents = _ints(case["parents"])
        keep = _ints(case["keep"]) if case["keep"] else [lens[p] for p in parents]
        most = {}
        for p, k in zip(parents, keep):
            most[p] = max(most.get(p, 0), _cdiv(k, page))
        return dict(bytes=4 * sum(_cdiv(k, page) for k in keep) + 12 * sum(most.values()) + 28 * len(parents), flops=0)
    pages = [_cdiv(x, page) for x in lens]
    if op == "trim":
        keep = _ints(case["keep"])
        gone = sum(max(0, p - _cdiv(k, page)) for p, k in zip(pages, keep))
        return dict(bytes=16 * gone + 12 * len(lens), flops=0)
    used = sum(pages) - sum(p * (n - 1) for p, n in _shared_pages(case))
    moved = used * (case["pool"] - case["to"]) // case["pool"]
    return dict(bytes=4 * sum(pages) + 8 * (case["pool"] - used) + 28 * moved + 4 * len(lens), flops=0)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    """Rows and caches in 64 bits, not rounded to the outputs' types; the page operators' outputs are whole numbers."""
    if case["op"] not in ("rope", "copy"):
        return None
    st = _prepare(case, _gen(seed))
    if case["op"] == "copy":
        pools = [st["cache"].double(), None if st["scales"] is None else st["scales"].double()]
        for s, d in zip(st["src"].tolist()[:case["pairs"]], st["dst"].tolist()):
            for x in pools:
                if x is not None:
                    x.select(2, d).copy_(x.select(2, s))
        return tuple(pools)
    r, page = case["rot"], case["page"]
    out = {}
    for name, x, w in (("q", st["q"], st["qw"]), ("k", st["k"], st["kw"])):
        y = x.double()
        if case["norm"]:
            y = y / torch.sqrt(torch.sum(y * y, -1, keepdim=True) / D + st["eps"]) * w.double()
        z = y.clone()
        for i in range(r // 2):
            a, b = (i, i + r // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
            turn = (st["pos"].double() * float(st["freq"][i]))[:, None]
            z[..., a] = y[..., a] * torch.cos(turn) - y[..., b] * torch.sin(turn)
            z[..., b] = y[..., a] * torch.sin(turn) + y[..., b] * torch.cos(turn)
        out[name] = z
    valid = st["pos"] >= 0
    q = torch.where(valid[:, None, None], out["q"], 0.0)
    if case["cache"] == "rows":
        return q, torch.where(valid[:, None, None], out["k"], 0.0), None, None
    kc, vc = st["kc"].double(), st["vc"].double()
    ks, vs = (st["ks"], st["vs"]) if case["cache"] == "e4m3" else (1.0, 1.0)
    tok = page or kc.shape[2]
    slots = st["slots"][valid]
    lead, off = torch.div(slots, tok, rounding_mode="floor"), torch.remainder(slots, tok)
    for cache, rows, s in ((kc, out["k"][valid], ks), (vc, st["v"][valid].double(), vs)):
        rows = (rows / s).clamp(-448, 448) if case["cache"] == "e4m3" else rows
        cache.transpose(1, 2)[lead, off] = rows
    return q, None, kc, vc
