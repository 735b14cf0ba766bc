"""Plain fp64 CPU oracle of accumulated attention weights and of eviction from the
paged cache.

TEST INFRASTRUCTURE ONLY, like kv_ref: nothing on the product path imports it,
and it shares no code with the CUDA path.  Weights are sums of exp(score - LSE)
over the query rows and heads of a group that see a key.  Eviction keeps, per
request and kv head, protected tokens first, then the heaviest, of equals the
lower row, and moves those from behind into the holes in front.
"""
from __future__ import annotations

import math

import torch

from oracle import attn_ref, kv_ref

F64 = torch.float64


def weigh(q, lse, cu, lens, table, kc, ke, weight, position, offsets, scale, mask=2, left=-1, right=-1, decay=1.0,
          new_lens=None):
    """New weights (fp64) and positions, and for tolerances the sum over the rows of
    p (ds + |s| + |LSE| + 1) units: see the tests.  weight and position [pages,
    heads, page] are not changed."""
    page, group = kc.shape[1], q.shape[1] // kc.shape[2]
    out, pos = weight.to(F64).clone(), position.clone()
    slack = torch.zeros_like(out)
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo or n == 0:
            continue
        pages = table[b][: (n + page - 1) // page]
        see = attn_ref.visible(hi - lo, n, mask, left, right)
        added = new_lens[b] if new_lens is not None else min(hi - lo, n) if mask in (2, 3) else 0
        touched = see.any(0) | (torch.arange(n) >= n - added) if decay == 1.0 else torch.ones(n, dtype=torch.bool)
        k = kv_ref.gather(kc, ke, [max(p, 0) for p in pages], n)
        for h in range(kc.shape[2]):
            got, err = torch.zeros(n, dtype=F64), torch.zeros(n, dtype=F64)
            for x in range(h * group, (h + 1) * group):
                qq, l = q[lo:hi, x].to(F64), lse[x, lo:hi].to(F64)[:, None]
                s = qq @ k[:, h].T * scale
                size = qq.abs() @ k[:, h].abs().T * abs(scale)
                p = torch.where(see & torch.isfinite(l), torch.exp(s - l), torch.zeros_like(s))
                got += p.sum(0)
                units = q.shape[2] * 2.0 ** -23 * size + 2.0 ** -22 * (s.abs() + l.abs() + 1)
                err += torch.where(p > 0, p * units, torch.zeros_like(p)).sum(0)
            for j in range(n):
                pg = pages[j // page]
                if pg < 0 or pg >= kc.shape[0] or not bool(touched[j]):
                    continue
                fresh = j >= n - added
                old = 0.0 if fresh or decay == 0.0 else decay * float(weight[pg, h, j % page])
                out[pg, h, j % page] = old + got[j]
                slack[pg, h, j % page] = err[j] + (2.0 ** -23 * ((hi - lo) * group + 8)) * (abs(old) + float(got[j]))
                if fresh:
                    pos[pg, h, j % page] = j + offsets[b]
    return out, pos, slack


def stays(weights, positions, keep, sink, first_recent):
    """The rows that stay: a list of `keep` row numbers, ascending."""
    def key(i):
        w = float(weights[i])
        protected = positions[i] < sink or positions[i] >= first_recent
        return (not protected, math.isnan(w), -w if not math.isnan(w) else 0.0, i)
    return sorted(sorted(range(len(weights)), key=key)[:keep])


def evict(keep, lens, offsets, table, free, free_count, cache, exps, weight, position, sink=0, recent=0, slack=0):
    """Lists and CPU tensors, changed in place (cache and exps: {k: ..., v: ...});
    returns (lens, offsets, free_count)."""
    page = weight.shape[2]
    lens, offsets = list(lens), list(offsets)
    for b, n in enumerate(lens):
        if keep[b] < 0 or n <= keep[b] + slack:
            continue
        to = keep[b]
        at = lambda row: (table[b][row // page], row % page)   # noqa: E731, B023
        for h in range(weight.shape[1]):
            w = [weight[at(i)[0], h, at(i)[1]] for i in range(n)]
            pos = [int(position[at(i)[0], h, at(i)[1]]) for i in range(n)]
            left = stays(w, pos, to, sink, n + offsets[b] - recent)
            there = set(left)
            pairs = list(zip([i for i in range(to) if i not in there], [i for i in left if i >= to]))
            for x in ("k", "v"):
                was = {i: (cache[x][at(i)[0], at(i)[1], h].clone(), kv_ref.clamp_exp(exps[x][at(i)[0], h])) for i in range(n)}
                for block in range((to + page - 1) // page):
                    here = [(d, s) for d, s in pairs if d // page == block]
                    if not here:
                        continue
                    pg = table[b][block]
                    old = was[block * page][1]
                    e = max([old] + [was[s][1] for _, s in here])
                    if e > old:
                        for i in range(block * page, min((block + 1) * page, to)):
                            cache[x][pg, i % page, h] = kv_ref.e4m3_byte(kv_ref.e4m3_value(was[i][0]) * 2.0 ** (old - e))
                        exps[x][pg, h] = e + 127
                    for d, s in here:
                        byte, es = was[s]
                        cache[x][pg, d % page, h] = byte if es == e else kv_ref.e4m3_byte(kv_ref.e4m3_value(byte) * 2.0 ** (es - e))
            moved = [(weight[at(s)[0], h, at(s)[1]].clone(), position[at(s)[0], h, at(s)[1]].clone()) for _, s in pairs]
            for (d, _), (x, y) in zip(pairs, moved):
                weight[at(d)[0], h, at(d)[1]] = x
                position[at(d)[0], h, at(d)[1]] = y
        for block in range((to + page - 1) // page, (n + page - 1) // page):
            free[free_count] = table[b][block]
            free_count += 1
        offsets[b] += n - to
        lens[b] = to
    return lens, offsets, free_count
