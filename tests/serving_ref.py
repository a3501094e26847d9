"""Plain 64-bit implementations of the serving operators (page tables, store
into a block-scaled E4M3 cache, decode over it, prompt attention), written from
their definitions for the tests.  They run wherever their inputs are."""
from __future__ import annotations

import math

import torch

D = 128
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ attention
def attend(q, k, v, seen):
    """q [n, D], k, v [m, D] in 64 bits, row i sees keys j < seen[i].
    Returns out, lse and the tolerance terms: a = sum_j w_j |v_j|, and per row
    the largest sum_d |q_d k_jd| / sqrt(D) and the largest |s| over its keys."""
    n, m = q.shape[0], k.shape[0]
    dev = q.device
    out = torch.zeros(n, D, dtype=torch.float64, device=dev)
    a = torch.zeros_like(out)
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
    absum = torch.zeros(n, dtype=torch.float64, device=dev)
    if m == 0 or n == 0:
        return out, lse, a, absum
    hidden = torch.arange(m, device=dev)[None, :] >= seen[:, None]
    s = (q @ k.T) / math.sqrt(D)
    s = torch.where(hidden, torch.full_like(s, -math.inf), s)
    some = seen > 0
    z = torch.logsumexp(s, 1)
    w = torch.exp(s - torch.where(some, z, torch.zeros_like(z))[:, None])
    # a hidden key's value has no part in the sum, whatever it is
    for i0 in range(0, n, 512):
        i1 = min(n, i0 + 512)
        top = int(seen[i0:i1].max())
        vv = v[:top]
        ww = w[i0:i1, :top]
        if not bool(torch.isfinite(vv).all()):
            for i in range(i0, i1):
                c = int(seen[i])
                out[i] = w[i, :c] @ v[:c] if c else 0
                a[i] = w[i, :c] @ v[:c].abs() if c else 0
            continue
        out[i0:i1] = ww @ vv
        a[i0:i1] = ww @ vv.abs()
    out[~some] = 0
    lse = torch.where(some, z, lse)
    ab = (q.abs() @ k.abs().T) / math.sqrt(D)
    absum = torch.where(hidden, torch.zeros_like(ab), ab).nan_to_num(0, 0, 0).amax(1)
    return out, lse, a, absum


def score_error(absum, n):
    """What 32-bit arithmetic may do to a row's weights, relative: the scores'
    128 products summed in 32 bits (128 * 2^-23 of their absolute sum; the
    tensor cores may truncate), the exponent's argument and reference (two
    roundings of at most |s| log2(e) each, |s| <= absum), the exponential (2^-22)
    and the sum of n weights (n 2^-24, taken for one thread adding them all)."""
    return absum * (2.0 ** -16 + 4 * 2.0 ** -23) + 2.0 ** -21 + n * 2.0 ** -24


def prompt(q, k, v, cu_q, cu_k, causal, out_dtype):
    """(out, lse, tolerance of out, tolerance of lse) of packed prompts; rows of
    no sequence are NaN in out and lse."""
    tq, hq, _ = q.shape
    G = hq // k.shape[1]
    u_p = torch.finfo(q.dtype).eps / 2        # the weights' rounding to the inputs' type
    u_o = torch.finfo(out_dtype).eps / 2
    out = torch.full((tq, hq, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((tq, hq), math.nan, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    tiny = 2.0 ** -133 if out_dtype == torch.bfloat16 else 2.0 ** -24 if out_dtype == torch.float16 else 2.0 ** -126
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        i = torch.arange(n, device=q.device)
        seen = (m - n + 1 + i).clamp(0, m) if causal else torch.full_like(i, m)
        for h in range(hq):
            qs = q[cu_q[b]:cu_q[b + 1], h].double()
            ks, vs = (x[cu_k[b]:cu_k[b + 1], h // G].double() for x in (k, v))
            o, z, a, ab = attend(qs, ks, vs, seen)
            e = score_error(ab, m)
            sl = slice(cu_q[b], cu_q[b + 1])
            out[sl, h], lse[sl, h] = o, z
            # weights and their sum both carry e; P is rounded once; so is out.
            # f16 weights below 2^-14 are off by up to 2^-25 absolute, of sums >= 2^-8
            # (the reference may lag the maximum by 2^8), beside m keys
            floor = 2.0 ** -17 * m * vs.abs().nan_to_num(0, 0, 0).max() if m and q.dtype == torch.float16 else 0.0
            tol[sl, h] = (u_p + 2 * e)[:, None] * a + u_o * o.abs() + tiny + 2.0 ** -8 * floor * 2.0 ** -8
            ltol[sl, h] = 2 * e + 2.0 ** -22 * z.abs().nan_to_num(0, 0, 0) + 2.0 ** -21
    return out, lse, tol, ltol


def dequantised(cache, scales, block):
    """[lead, H, tokens, D] in 64 bits of a stored cache and its scales [lead, H, n]."""
    x = cache.double()
    s = scales.double().repeat_interleave(block, 2)[:, :, :x.shape[2]]
    return x * s[..., None]


def decode(q, kc, vc, ks, vs, block, lens, table, page, out_dtype, k_scale=1.0, v_scale=1.0):
    """q [B, q_len, Hq, D]; (out, lse, tolerances)."""
    B, ql, hq, _ = q.shape
    hkv = kc.shape[1]
    G = hq // hkv
    u_o = torch.finfo(out_dtype).eps / 2
    out = torch.zeros(B, ql, hq, D, dtype=torch.float64, device=q.device)
    lse = torch.zeros(B, ql, hq, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    kd, vd = dequantised(kc, ks, block) * k_scale, dequantised(vc, vs, block) * v_scale
    for b in range(B):
        n = int(lens[b])
        t = torch.arange(n, device=q.device)
        lead, off = (table[b].long()[t // page], t % page) if page else (torch.full_like(t, b), t)
        seen = (n - ql + 1 + torch.arange(ql, device=q.device)).clamp(min=0).repeat_interleave(G)
        for h in range(hkv):
            qs = q[b, :, h * G:(h + 1) * G].reshape(-1, D).double()
            o, z, a, ab = attend(qs, kd[lead, h, off], vd[lead, h, off], seen)
            # the scales add a product and, as log2, an addend of at most 2^7 rounded
            # to 32 bits, and the weights are carried to 2^-21; the split states are
            # joined in 32 bits (a sum of up to 128)
            e = score_error(ab, n) + 2.0 ** -16 + 2.0 ** -17
            tol[b, :, h * G:(h + 1) * G] = ((2 * e + 2.0 ** -17)[:, None] * a + u_o * o.abs() + 2.0 ** -24).view(ql, G, D)
            ltol[b, :, h * G:(h + 1) * G] = (2 * e + 2.0 ** -22 * z.abs().nan_to_num(0, 0, 0)).view(ql, G)
            out[b, :, h * G:(h + 1) * G] = o.view(ql, G, D)
            lse[b, :, h * G:(h + 1) * G] = z.view(ql, G)
    return out, lse, tol, ltol


def close(got, want, tol, what):
    """|got - want| <= tol where want is finite; infinities and NaN at the same places."""
    got, want = got.double(), want.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: finite at other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    err = torch.where(fin, (got - want).abs(), torch.zeros_like(want))
    bad = err > tol
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {err.max().item():.3e}, "
                                 f"{(err / tol.clamp(min=1e-300)).max().item():.2f} of its tolerance")


# ------------------------------------------------------------------ store
def e4m3_values():
    """The 127 non-negative E4M3 values."""
    return torch.arange(127, dtype=torch.uint8).view(F8).double()


def to_e4m3(x):
    """Nearest E4M3 value (ties to even mantissa) of 64-bit x, |x| <= 448 or NaN, by search in the table."""
    vals = e4m3_values().to(x.device)
    a = x.abs().nan_to_num(0.0)
    hi = torch.searchsorted(vals, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - vals[lo], vals[hi] - a
    pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    y = torch.copysign(vals[pick], x)
    return torch.where(torch.isnan(x), torch.full_like(y, math.nan), y)


def store(new, slots, cache, scales, row_tokens, block):
    """(values, scales) in 64 bits after storing rows new [n, H, D] (see fd_cache_store)."""
    c, s = cache.double().clone(), scales.double().clone()
    n = new.shape[0]
    sl = slots.tolist()
    t = 0
    n_slots = cache.shape[0] * row_tokens
    while t < n:
        if sl[t] < 0 or sl[t] >= n_slots:
            t += 1
            continue
        lead, off = divmod(sl[t], row_tokens)
        row0, blk = off % block, off // block
        # the rows that follow in the block, at their distance; skipped ones between them have no part
        rows, d = [0], 1
        while t + d < n and row0 + d < block and off + d < row_tokens:
            if 0 <= sl[t + d] < n_slots:
                if sl[t + d] != sl[t] + d:
                    break
                rows.append(d)
            d += 1
        r = torch.tensor(rows, device=new.device)
        x = new[t:t + d].double()[r].transpose(0, 1)                     # [H, rows, D]
        x = torch.where(torch.isfinite(x), x, torch.full_like(x, math.nan))
        big = x.abs().nan_to_num(0.0).amax((1, 2))
        for h in range(new.shape[1]):
            need = -126
            while 448.0 * 2.0 ** need < float(big[h]):
                need += 1
            need = 2.0 ** need
            was = float(s[lead, h, blk])
            now = need if row0 == 0 else max(was, need)
            if row0 and now != was:
                c[lead, h, off - row0:off] = to_e4m3(c[lead, h, off - row0:off] * (was / now))
            c[lead, h, off + r] = to_e4m3(x[h] / now)
            s[lead, h, blk] = now
        t += rows[-1] + 1
    return c, s


# ------------------------------------------------------------------ tables
def tables(lens, new, free, count, table, page, n_pages, n_slots):
    """The outputs of fd_page_tables on host lists: (lens, count, table, cu, slots, positions, bad)."""
    width = len(table[0]) if table else 0
    table = [list(r) for r in table]
    lens_out, slots, pos = list(lens), [-1] * n_slots, [-1] * n_slots
    bad = not 0 <= count <= len(free)
    count = min(max(count, 0), len(free))
    cu, tok, want, taken = [0], 0, 0, 0
    for b, (held, n) in enumerate(zip(lens, new)):
        ok = held >= 0 and n >= 0 and held + n <= width * page
        n = max(n, 0)
        ok = ok and tok + n <= n_slots
        if ok:
            have, last = -(-held // page), -(-(held + n) // page)
            want += last - have
            ok = last == have or want <= count
            if ok and last > have:
                for i in range(have, last):
                    table[b][i] = free[count - 1 - (want - (last - have) + i - have)]
                taken = want
        bad = bad or not ok
        for i in range(n):
            if tok + i < n_slots:
                pos[tok + i] = held + i
                if ok:
                    pg = table[b][(held + i) // page]
                    if 0 <= pg < n_pages:
                        slots[tok + i] = pg * page + (held + i) % page
                    else:
                        bad = True
        if ok:
            lens_out[b] = held + n
        tok += n
        cu.append(tok)
    return lens_out, count - taken, table, cu, slots, pos, bad
