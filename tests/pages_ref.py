"""Plain implementations of fd_page_fork, fd_page_trim, fd_page_compact (lists of
whole numbers, one step after another, from their definitions) and of fd_qkv_rope
(64 bits), for the tests.  The page functions return what the call leaves in
its buffers and whether it has something to report."""
from __future__ import annotations

import math

import torch

D = 128
F8 = torch.float8_e4m3fn


def fork(parents, children, keep, lens, free, count, table, shares, page, n_pages, src, dst):
    width = len(table[0]) if table else 1
    bad = not 0 <= count <= len(free)
    count = min(max(count, 0), len(free))
    lens_out, table, shares = list(lens), [list(r) for r in table], list(shares)
    src, dst = list(src), list(dst)
    n, owner = 0, {}
    for i, (a, b) in enumerate(zip(parents, children)):
        ok = 0 <= a < len(lens) and 0 <= b < len(lens) and a != b
        if ok:
            k = lens[a] if keep is None else keep[i]
            ok = 0 <= lens[a] <= width * page and lens[b] == 0 and 0 <= k <= lens[a] and b not in owner
        if not ok:
            bad = True
            continue
        owner[b] = i
        full, part = k // page, k % page != 0
        if part and n >= count:
            bad = True
            continue
        for j in range(full):
            p = table[a][j]
            table[b][j] = p
            if 0 <= p < n_pages:
                shares[p] += 1
            else:
                bad = True
        if part:
            new, old = free[count - 1 - n], table[a][full]
            bad |= not (0 <= new < n_pages and 0 <= old < n_pages)
            table[b][full] = new
            src[n], dst[n] = old, new
            n += 1
        lens_out[b] = k
    return dict(lens=lens_out, count=count - n, table=table, shares=shares, free=list(free), src=src, dst=dst, n=n), bad


def trim(keep, lens, free, count, table, shares, page, n_pages, src, dst):
    B = len(lens)
    width = len(table[0]) if table else 1
    bad = not 0 <= count <= len(free)
    count = min(max(count, 0), len(free))
    table, free = [list(r) for r in table], list(free)
    given = shares is not None
    shares = list(shares) if given else [0] * n_pages
    before = list(shares)
    src, dst = list(src), list(dst)
    plan, need = [], 0                   # tokens kept, or None: left as it is
    for b in range(B):
        k = keep[b]
        if not 0 <= lens[b] <= width * page:
            bad, k = True, None
        elif k < 0 or k >= lens[b]:
            k = None
        tail = None
        if k is not None and k % page and given:
            tail = table[b][k // page]
            if not 0 <= tail < n_pages:
                bad, tail = True, None
        if tail is not None and before[tail] > 0:
            need += 1
            if need > count:
                bad, k, tail = True, None, None
        plan.append((k, tail))
    holders, events = {}, {}             # page -> what becomes of it
    order = []
    for b, (k, tail) in enumerate(plan):
        if k is None:
            continue
        for j in range(-(-k // page), -(-lens[b] // page)):
            p = table[b][j]
            if not 0 <= p < n_pages:
                bad = True
                continue
            order.append(p)
            events.setdefault(p, [0, []])[0] += 1
        if tail is not None:
            events.setdefault(tail, [0, []])[1].append(b)
    moves, back = set(), set()
    for p, (gone, claims) in events.items():
        left = shares[p] + 1 - gone - len(claims) if given else 0
        if left < 0:
            bad = True
        if left > 0:
            moves.update(claims)
            shares[p] = left - 1
        else:
            shares[p] = 0
            if claims:
                moves.update(claims[:-1])
            else:
                back.add(p)
    n = 0
    for b in sorted(moves):
        k, tail = plan[b]
        new = free[count - 1 - n]
        bad |= not 0 <= new < n_pages
        src[n], dst[n] = tail, new
        table[b][k // page] = new
        n += 1
    if given:                            # a page goes back at the last place in the order
        last = {p: i for i, p in enumerate(order)}
        given_back = [p for i, p in enumerate(order) if p in back and last[p] == i]
    else:
        given_back = list(order)
    base = count - n
    for i, p in enumerate(given_back):
        at = base + len(given_back) - 1 - i
        if at < len(free):
            free[at] = p
        else:
            bad = True
    return dict(lens=[lens[b] if plan[b][0] is None else plan[b][0] for b in range(B)], count=min(base + len(given_back), len(free)),
                table=table, shares=shares if given else None, free=free, src=src, dst=dst, n=n), bad


def compact(n_keep, lens, free, count, table, shares, page, n_pages, src, dst):
    width = len(table[0]) if table else 1
    bad = not 0 <= count <= len(free)
    count = min(max(count, 0), len(free))
    table, free, src, dst = [list(r) for r in table], list(free), list(src), list(dst)
    shares = None if shares is None else list(shares)
    live = []
    for b, x in enumerate(lens):
        if not 0 <= x <= width * page:
            bad = True
            continue
        live += [(b, j) for j in range(-(-x // page))]
    held = set()
    for b, j in live:
        p = table[b][j]
        if not 0 <= p < n_pages:
            bad = True
        elif p >= n_keep:
            held.add(p)
    bad |= any(not 0 <= p < n_pages for p in free[:count])
    F = [p for p in free[:count] if 0 <= p < n_keep]
    m = min(len(held), len(F), len(src))
    bad |= m < len(held)
    names = {p: F[len(F) - 1 - i] for i, p in enumerate(sorted(held)[:m])}
    for b, j in live:
        table[b][j] = names.get(table[b][j], table[b][j])
    for i, (p, q) in enumerate(names.items()):
        src[i], dst[i] = p, q
        if shares is not None:
            shares[q], shares[p] = shares[p], 0
    free[:len(F)] = F
    return dict(count=len(F) - m, table=table, shares=shares, free=free, src=src, dst=dst, n=m), bad


def rope(x, w, norm, pos, inv_freq, rot, interleaved, eps, rot_scale):
    """Rows x [n, heads, D] normed and rotated in 64 bits, and what 32-bit arithmetic may
    be off by, element by element (before the result's own rounding).

    Norm: a sum of 128 products (16 in one lane, then three levels: 19 roundings
    and the squares' own, of a sum of positive numbers: 20 u relative, halved by
    the root), mean and eps (2 u, halved), the reciprocal root (2 ulp = 4 u), the
    products with it and with w (2 u): 18 u taken, u = 2^-24.
    Rotation: the angle is off by half a step of a 32-bit fraction in [-1, 1) half
    turns (2^-25 of pi), the cut at 2^-32 of a turn and inv_freq / 2 pi's 2^-62 part per
    position (far less): 1.2e-7 radians taken; sine and cosine to 2 ulp (of 1: 4 u), their product
    with the scale u: in all 2^-23 + 5 u + ... < 8 u of the scale each.  Two products and a
    sum: 2 u of the magnitudes.  So 12 u (|a| + |b|) |scale| covers the turn."""
    u = 2.0 ** -24
    y = x.double()
    err = torch.zeros_like(y)
    if norm:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + eps)
        if w is not None:
            y = y * w.double()
        err = 18 * u * y.abs()
    z, e = y.clone(), err.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = pos.double() * float(inv_freq[i])
        c, s = (f(t)[:, None] * rot_scale for f in (torch.cos, torch.sin))
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        both = (err[..., a] + err[..., b] + 12 * u * (y[..., a].abs() + y[..., b].abs())) * abs(rot_scale)
        e[..., a] = both
        e[..., b] = both
    return z, e


def rounding(y, dtype):
    """Half a step of the output type at y (bounded from above), its smallest step included."""
    tiny = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, F8: 2.0 ** -10}[dtype]
    return y.abs() * (torch.finfo(dtype).eps / 2) + tiny


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: finite at other places"
    err = torch.where(fin, (got - want).abs(), torch.zeros_like(want))
    bad = err > tol
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {err.max().item():.3e}, "
                                 f"{(err / tol.clamp(min=1e-300)).max().item():.2f} of its tolerance")


def inv_freq(theta, rot):
    return torch.tensor([1.0 / theta ** (2 * i / rot) for i in range(rot // 2)], dtype=torch.float32)


assert math.isclose(float(inv_freq(10000.0, 64)[0]), 1.0)
