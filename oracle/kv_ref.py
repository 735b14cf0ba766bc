"""Plain fp64 CPU oracle of rotary positions and the paged 8-bit cache.

TEST INFRASTRUCTURE ONLY, like attn_ref: nothing on the product path imports
it, and it shares no code with the CUDA path.  Definitions:

* rope: pair (a, b) of a row becomes (a cos t - b sin t, b cos t + a sin t),
  t = positions[pair_axis[i]] * inv_freq[i]; pairs are (i, i + rot / 2) or
  (2 i, 2 i + 1); the other columns stay.
* cache: e4m3 values (sign, 4 exponent bits with bias 7, 3 mantissa bits, no
  infinities, largest 448) times 2^(byte - 127) per page and head.  Appending a
  run of tokens to a page sets or raises the scale to the least power of two
  that holds the run's largest finite magnitude, and rounds the rows in front of the
  run again when it grew.
* plan: the page stack and block tables of the C header, one page at a time.
* attention over the cache: attn_ref's forward on each request's gathered,
  dequantised keys and values.
"""
from __future__ import annotations

import math

import torch

from oracle import attn_ref

F64 = torch.float64


def rope(x, positions, inv_freq, pair_axis=None, interleaved=False, inverse=False):
    """x [rows, heads, d] in float64, positions [axes, rows]."""
    y = x.to(F64).clone()
    half = inv_freq.numel()
    for i in range(half):
        ax = 0 if pair_axis is None else int(pair_axis[i])
        t = positions[ax].to(F64) * float(inv_freq[i])
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        s = -s if inverse else s
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        xa, xb = x[..., a].to(F64), x[..., b].to(F64)
        y[..., a] = xa * c - xb * s
        y[..., b] = xb * c + xa * s
    return y


# ---------------------------------------------------------------------- e4m3

def _e4m3_table():
    vals = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v = math.nan if (b & 127) == 127 else v
        vals.append(-v if b & 128 else v)
    return torch.tensor(vals, dtype=F64)


E4M3 = _e4m3_table()


def e4m3_value(byte):
    return E4M3[byte.to(torch.int64)]


def e4m3_byte(x):
    """Nearest e4m3 byte (ties to the even mantissa, beyond 448 clamped, NaN 0x7f)."""
    x = x.to(F64)
    mags = E4M3[:127]                                   # ascending, 0 .. 448
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(mags, a).clamp(max=126)     # first magnitude >= a
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - mags[lo], mags[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    out = pick + torch.where(torch.signbit(x), 128, 0)
    return torch.where(torch.isnan(x), 127, out).to(torch.uint8)


def exponent_for(amax):
    """Least e in [-30, 30] with amax <= 448 * 2^e."""
    e = -30
    while e < 30 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def clamp_exp(byte):
    return max(-30, min(30, int(byte) - 127))


def append(cache, exps, x, slots):
    """In place: cache uint8 [pages, page, heads, d], exps uint8 [pages, heads],
    x [tokens, heads, d], slots list.  The tokens of one page form a run; rows
    in front of its first row are live."""
    pages, page = cache.shape[:2]
    x = x.to(F64)
    by_page = {}
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            by_page.setdefault(s // page, []).append((t, s % page))
    for p, run in by_page.items():
        toks, rows = [t for t, _ in run], [r for _, r in run]
        r = min(rows)
        for h in range(x.shape[1]):
            part = x[toks, h]
            mags = part.abs()[torch.isfinite(part)]
            e = exponent_for(float(mags.max()) if mags.numel() else 0.0)
            if r > 0:
                old = clamp_exp(exps[p, h])
                e = max(e, old)
                if e > old:
                    cache[p, :r, h] = e4m3_byte(e4m3_value(cache[p, :r, h]) * 2.0 ** (old - e))
            cache[p, rows, h] = e4m3_byte(part * 2.0 ** -e)
            exps[p, h] = e + 127


def plan(new_lens, seqlens, table, free, free_count, page, max_tokens):
    """Lists in; (cu, seqlens, positions, slots, free_count), with table (list of
    lists) and free (list, changed in place)."""
    count = lambda n: (n + page - 1) // page   # noqa: E731
    for b, n in enumerate(new_lens):
        if n < 0:
            for j in range(count(seqlens[b])):
                free[free_count] = table[b][j]
                free_count += 1
    cu, after, pos, slots = [0], [], [], []
    for b, n in enumerate(new_lens):
        was = 0 if n < 0 else seqlens[b]
        n = max(n, 0)
        for j in range(count(was), count(was + n)):
            free_count -= 1
            table[b][j] = free[free_count]
        after.append(was + n)
        cu.append(cu[-1] + n)
        for i in range(was, was + n):
            pos.append(i)
            slots.append(table[b][i // page] * page + i % page)
    pos += [0] * (max_tokens - len(pos))
    slots += [-1] * (max_tokens - len(slots))
    return cu, after, pos, slots, free_count


def gather(cache, exps, pages, n):
    """The first n tokens of these pages, dequantised: [n, heads, d]."""
    parts = [e4m3_value(cache[p]) * torch.tensor([2.0 ** clamp_exp(b) for b in exps[p]], dtype=F64)[None, :, None]
             for p in pages]
    return torch.cat(parts)[:n] if parts else torch.zeros((0,) + tuple(cache.shape[2:]), dtype=F64)


def attend(q, cu, lens, table, kc, vc, ke, ve, scale, mask=0, left=-1, right=-1):
    """O [T, Hq, d_v], LSE [Hq, T] and, for tolerances, the weighted mean
    magnitude sum p |v| / l [T, Hq, d_v] and the largest sum |q k| scale of a
    row's keys [Hq, T].  Rows of no segment: NaN."""
    page, group = kc.shape[1], q.shape[1] // kc.shape[2]
    o = torch.full(q.shape[:2] + (vc.shape[3],), math.nan, dtype=F64)
    mag = torch.zeros_like(o)
    lse = torch.full((q.shape[1], q.shape[0]), math.nan, dtype=F64)
    size = torch.zeros_like(lse)
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        pages = table[b][: (n + page - 1) // page]
        k, v = gather(kc, ke, pages, n), gather(vc, ve, pages, n)
        see = attn_ref.visible(hi - lo, n, mask, left, right)
        for h in range(q.shape[1]):
            qq, kk, vv = q[lo:hi, h].to(F64), k[:, h // group], v[:, h // group]
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            any_key = see.any(1)
            m = s.max(1, keepdim=True).values if n else torch.full((hi - lo, 1), -math.inf, dtype=F64)
            p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
            l = p.sum(1, keepdim=True)
            one = torch.where(l == 0, torch.ones_like(l), l)
            o[lo:hi, h] = p @ vv / one
            mag[lo:hi, h] = p @ vv.abs() / one
            lse[h, lo:hi] = torch.where(any_key, (m + l.log())[:, 0], torch.full_like(m[:, 0], -math.inf))
            if n:
                size[h, lo:hi] = (qq.abs() @ kk.abs().T).max(1).values * abs(scale)
    return o, lse, mag, size
