"""Operators for what attention keeps in eight bits, with their plain forms.

Two for training, two for serving:

* checkpoint: q, k, v and o of a forward pass as 8-bit whole numbers with one
  power-of-two scale per 32 columns, half the memory until the backward pass;
* attn_backward_checkpoint: dq, dk and dv from such a checkpoint;
* kv_weigh: the attention weight that every cached token of a paged cache gets
  from the new tokens, added to what it has got so far;
* kv_evict: per request and kv head, the tokens with the largest weights stay,
  the holes in front are filled from behind, the pages left over are given back.

`listed()` names the measured cases, `draw()` gives more of the same ranges.
`run(state)` makes one pass: with `own` false in elementary torch operations in
32 bits, with `own` true through this package's entry points.  `exact(case,
seed)` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

F64, F32, I32, I64 = torch.float64, torch.float32, torch.int32, torch.int64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MASKS = {"none": 0, "top_left": 1, "causal": 2, "window": 3}      # attn_mask_t
GROUP = 32                        # columns that share a scale
EXP_BIAS, EXP_MIN = 127, -126     # scale of a group, and of a cache page and head: 2^(byte - 127)
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one layer of a short sequence: the smallest call, all latency
        dict(name="checkpoint_small", op="checkpoint", batch=1, lo=333, hi=333, packed=False, hq=8, hkv=8, dqk=64, dv=64,
             dtype="fp16"),
        # packed sequences, unequal head dims
        dict(name="checkpoint_packed", op="checkpoint", batch=4, lo=7, hi=1801, packed=True, hq=16, hkv=4, dqk=192,
             dv=128, dtype="bf16"),
        # one layer of a training batch: memory bandwidth
        dict(name="checkpoint_train", op="checkpoint", batch=2, lo=4096, hi=4096, packed=False, hq=32, hkv=8, dqk=128, dv=128,
             dtype="bf16"),
        # short odd sequences: latency
        dict(name="backward_small", op="backward", batch=2, lo=129, hi=129, packed=False, hq=4, hkv=2, dqk=64, dv=64,
             mask="top_left", left=-1, dtype="fp16"),
        # packed sequences of different lengths, one very short
        dict(name="backward_packed", op="backward", batch=9, lo=1, hi=4001, packed=True, hq=16, hkv=4, dqk=128,
             dv=128, mask="top_left", left=-1, dtype="bf16"),
        # one layer of a training batch: compute
        dict(name="backward_train", op="backward", batch=2, lo=4096, hi=4096, packed=False, hq=32, hkv=8, dqk=128, dv=128,
             mask="top_left", left=-1, dtype="bf16"),
        # one token each of a small chat batch: latency
        dict(name="weigh_small", op="weigh", batch=4, page=16, lo=700, hi=1025, new=1, hq=32, hkv=8, dqk=128, dv=128,
             mask="causal", left=-1, decay=1.0, dtype="bf16"),
        # a full decode batch of ragged contexts: cache bandwidth
        dict(name="weigh_batch", op="weigh", batch=64, page=16, lo=500, hi=8192, new=1, hq=32, hkv=8, dqk=128, dv=128,
             mask="causal", left=-1, decay=1.0, dtype="bf16"),
        # prompt pieces behind a cached prefix: compute
        dict(name="weigh_prompt", op="weigh", batch=4, page=16, lo=3500, hi=5120, new=1024, hq=32, hkv=8, dqk=128,
             dv=128, mask="causal", left=-1, decay=1.0, dtype="bf16"),
        # decoding at a budget of 2,048 tokens: up to 64 too many, evicted many times before
        dict(name="evict_step", op="evict", batch=32, page=16, lo=2049, hi=2112, keep=2048, sink=4, recent=256,
             past=3000, hkv=8, dqk=128, dv=128),
        # after ragged prompts: a quarter of the longest one stays
        dict(name="evict_prompt", op="evict", batch=9, page=32, lo=1500, hi=8100, keep=2025, sink=4, recent=64, past=0,
             hkv=4, dqk=192, dv=128),
        # one very long context
        dict(name="evict_long", op="evict", batch=1, page=64, lo=131072, hi=131072, keep=32768, sink=16, recent=1024,
             past=0, hkv=8, dqk=128, dv=128),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


DIMS = ((64, 64), (128, 128), (192, 128), (256, 256))


def draw(rng):
    op = rng.choice(("checkpoint", "backward", "weigh", "evict"))
    dqk, dv = rng.choice(DIMS)
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
    if op in ("checkpoint", "backward"):
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        if dtype == "fp32":
            dqk, dv = rng.choice((32, 64)), rng.choice((32, 64))
        hkv, group = rng.choice((1, 2, 4)), rng.choice((1, 2, 3, 4))
        packed = rng.random() < 0.5
        top = 512 if dtype == "fp32" and op == "backward" else 4000
        batch = rng.randint(1, 7)
        hi = _spread(rng, 1, max(2, top // batch))
        c = dict(op=op, batch=batch, lo=rng.randint(0, hi) if packed else hi, hi=hi, packed=packed, hq=hkv * group, hkv=hkv, dqk=dqk, dv=dv, dtype=dtype)
        if op == "backward":
            mask = rng.choice(("none", "top_left", "causal", "window"))
            c.update(mask=mask, left=_spread(rng, 1, hi) if mask == "window" else -1)
        return c
    batch, page = _spread(rng, 1, 64), rng.choice((16, 32, 64, 128))
    if op == "weigh":
        new = 1 if rng.random() < 0.4 else _spread(rng, 2, max(3, 1000 // batch))
        hi = _spread(rng, new + 1, max(new + 2, min(16384, 100000 // batch)))
        mask = rng.choice(("none", "causal", "causal", "window"))
        return dict(op=op, batch=batch, page=page, lo=rng.randint(0, hi), hi=hi, new=new, hq=hkv * group, hkv=hkv,
                    dqk=dqk, dv=dv, mask=mask, left=_spread(rng, 1, hi) if mask == "window" else -1,
                    decay=rng.choice((1.0, 1.0, 0.9, 0.0)), dtype=rng.choice(("bf16", "fp16")))
    hi = _spread(rng, 2, max(3, 60000 // batch))
    return dict(op=op, batch=batch, page=page, lo=rng.randint(0, hi), hi=hi, keep=rng.randint(0, hi),
                sink=rng.randint(0, 8), recent=_spread(rng, 1, max(2, hi // 4)),
                past=rng.choice((0, rng.randint(1, 500))), hkv=hkv, dqk=dqk, dv=dv)


def _lengths(n, lo, hi):
    """n lengths spread over [lo, hi] that depend on nothing but these numbers, hi among them."""
    return [hi if i == 0 else lo + ((i * 2654435769 % 2 ** 32) * (hi - lo + 1) >> 32) for i in range(n)]


def _lens(c):
    """Lengths of the sequences of a training batch."""
    return _lengths(c["batch"], c["lo"], c["hi"])


def _new(c):
    """New tokens of every request of a weigh call."""
    return [c["new"] if i % 3 != 1 else max(1, c["new"] - (i * 31) % c["new"]) for i in range(c["batch"])]


def _pages(tokens, page):
    return (tokens + page - 1) // page


# ------------------------------------------------------------------ inputs

def _shape(c):
    """Leading dimensions of a tensor of the training side: [T] or [B, S]."""
    return (sum(_lens(c)),) if c["packed"] else (c["batch"], c["hi"])


def _parts(c, *tensors):
    """Per sequence, the [rows, heads, d] views of these tensors."""
    at = 0
    for b, n in enumerate(_lens(c)):
        yield [x[at:at + n] if c["packed"] else x[b] for x in tensors]
        at += n


def _seen(mask, left, lq, lk, dev):
    """[lq, lk]: which key each query sees (bottom-right causal and window look back from the end)."""
    i = torch.arange(lq, device=dev)[:, None]
    j = torch.arange(lk, device=dev)
    if mask == "none":
        return torch.ones((lq, lk), dtype=torch.bool, device=dev)
    if mask != "top_left":
        i = i + (lk - lq)
    see = j <= i
    return see & (j >= i - left) if mask == "window" else see


def _table(lens, page, spare, g, dev):
    """Block table of requests with these lengths, its pages in random order, and the pool's size."""
    need = [_pages(x, page) for x in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g, device=dev).to(I32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=I32, device=dev)
    at = torch.arange(table.shape[1], device=dev)
    table[at < torch.tensor(need, device=dev)[:, None]] = order[: sum(need)]
    return table, order, pool


def _cache(pool, page, hkv, d, g, dev):
    """A filled cache half: e4m3 values of a normal distribution and the exponents of their pages and heads."""
    x = torch.empty((pool, page, hkv, d), dtype=torch.float8_e4m3fn, device=dev)
    for i in range(0, pool, 8192):   # in parts: the 32-bit draws are four times the cache
        part = torch.randn(x[i:i + 8192].shape, generator=g, device=dev)
        x[i:i + 8192] = part.mul_(110).clamp_(-E4M3_MAX, E4M3_MAX).to(x.dtype)
    e = torch.randint(EXP_BIAS - 8, EXP_BIAS - 5, (pool, hkv), generator=g, device=dev, dtype=torch.uint8)
    return x, e


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES.get(c.get("dtype"))
    s = {"case": c}
    if c["op"] in ("checkpoint", "backward"):
        # heads of activations differ in size, and a few columns stand out
        rand = lambda h, d: (torch.randn((*_shape(c), h, d), generator=g, device=dev)   # noqa: E731
                             * torch.rand((h, d), generator=g, device=dev).mul(1.5).add(0.5)).to(dt)
        q, k, v = rand(c["hq"], c["dqk"]), rand(c["hkv"], c["dqk"]), rand(c["hkv"], c["dv"])
        if c["op"] == "checkpoint":
            return {**s, "q": q, "k": k, "v": v, "o": rand(c["hq"], c["dv"])}
        s["do"] = torch.randn((*_shape(c), c["hq"], c["dv"]), generator=g, device=dev).to(dt)
        if c["packed"]:
            s["cu_seqlens"] = torch.tensor([0] + _lens(c), dtype=I64).cumsum(0).to(dev, I32)
        # the forward pass, in elementary operations
        o, lse, group = torch.empty_like(s["do"]), [], c["hq"] // c["hkv"]
        for qs, ks, vs, os in _parts(c, q, k, v, o):
            hide = ~_seen(c["mask"], c["left"], qs.shape[0], qs.shape[0], dev)
            rows = []
            for h in range(c["hkv"]):
                sc = torch.einsum("qgd,kd->gqk", qs[:, h * group:(h + 1) * group].to(F32), ks[:, h].to(F32))
                sc.mul_(_softmax_scale(c)).masked_fill_(hide, -math.inf)
                rows.append(sc.logsumexp(-1))
                p = sc.sub_(rows[-1].masked_fill(rows[-1] == -math.inf, 0.0)[..., None]).exp_()
                os[:, h * group:(h + 1) * group] = torch.einsum("gqk,kd->qgd", p, vs[:, h].to(F32)).to(dt)
            lse.append(torch.cat(rows))
        s["lse"] = torch.cat(lse, 1) if c["packed"] else torch.stack(lse)
        for n, x in (("q", q), ("k", k), ("v", v), ("o", o)):
            s[n], s[n + "_exp"] = _quantised(x)
        return s
    after = _lengths(c["batch"], c["lo"], c["hi"])
    page, hkv = c["page"], c["hkv"]
    if c["op"] == "weigh":
        new = _new(c)
        after = [max(a, n) for a, n in zip(after, new)]
    table, order, pool = _table(after, page, 5, g, dev)
    s["block_table"], s["seqlens"] = table, torch.tensor(after, dtype=I32, device=dev)
    s["k_cache"], s["k_exp"] = _cache(pool, page, hkv, c["dqk"], g, dev)
    s["v_cache"], s["v_exp"] = _cache(pool, page, hkv, c["dv"], g, dev)
    s["status"] = torch.zeros(1, dtype=I32, device=dev)
    # attention weights are spread over several orders of magnitude
    s["weight"] = (2 * torch.randn((pool, hkv, page), generator=g, device=dev)).exp_()
    s["position"] = torch.zeros((pool, hkv, page), dtype=I32, device=dev)
    past = torch.full((c["batch"],), c.get("past", 0), dtype=I32, device=dev)
    if c["op"] == "weigh":
        cu = torch.tensor([0] + new, dtype=I64).cumsum(0)
        s["cu_seqlens"], s["position_offsets"] = cu.to(dev, I32), past
        s["q"] = torch.randn((sum(new), c["hq"], c["dqk"]), generator=g, device=dev).to(dt)
        s["lse"] = torch.empty((c["hq"], sum(new)), device=dev)
        for b in range(c["batch"]):
            sc = _request_scores(s, c, b, cu.tolist(), after[b], F32)
            s["lse"][:, cu[b]:cu[b + 1]] = sc.logsumexp(-1).flatten(0, 1)
        return s
    # positions: as appended, or, after earlier evictions, in any order
    for b, n in enumerate(after):
        at = (torch.arange(n, device=dev).expand(hkv, n) if c["past"] == 0 else
              torch.rand((hkv, n + c["past"]), generator=g, device=dev).argsort(-1)[:, :n])
        i = torch.arange(n, device=dev)
        s["position"][table[b, i // page].to(I64), :, i % page] = at.T.to(I32)
    used = sum(_pages(x, page) for x in after)
    s["free_pages"] = torch.zeros(pool, dtype=I32, device=dev)
    s["free_pages"][: pool - used] = order[used:]
    s["free_count"] = torch.tensor([pool - used], dtype=I32, device=dev)
    s["position_offsets"] = past
    s["keep"] = torch.full((c["batch"],), c["keep"], dtype=I32, device=dev)
    return s


# ------------------------------------------------------------- plain forms

def _softmax_scale(c):
    return 1.0 / math.sqrt(c["dqk"])


def _quantised(x):
    """x in whole numbers of -127 .. 127 times a power of two per 32 columns, the least that holds them."""
    y = x.to(F32).unflatten(-1, (-1, GROUP))
    amax = y.abs().amax(-1)
    m, k = torch.frexp(amax)                     # amax = m 2^k, 0.5 <= m < 1; 127 = 0.9921875 * 2^7
    e = k - 7 + (m > 0.9921875).to(k.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)
    whole = torch.ldexp(y, -e[..., None]).round_().to(torch.int8).flatten(-2)
    return whole, (e + EXP_BIAS).to(torch.uint8)


def _values(whole, exp, dtype):
    """What a checkpoint's numbers stand for, in the type that they came from."""
    y = torch.ldexp(whole.to(F32).unflatten(-1, (-1, GROUP)), (exp.to(I32) - EXP_BIAS)[..., None])
    top = torch.finfo(dtype).max
    return y.flatten(-2).clamp(-top, top)


def _plain_checkpoint(s, c):
    out = {}
    for n in ("q", "k", "v", "o"):
        out[n], out[n + "_exp"] = _quantised(s[n])
    return out


def _plain_backward(s, c):
    dt, scale, group = s["do"].dtype, _softmax_scale(c), c["hq"] // c["hkv"]
    q, k, v, o = (_values(s[n], s[n + "_exp"], dt) for n in ("q", "k", "v", "o"))
    dq, dk, dv = (torch.empty(x.shape, dtype=dt, device=x.device) for x in (q, k, v))
    lses = s["lse"].split(_lens(c), 1) if c["packed"] else s["lse"]
    for (qs, ks, vs, os, ds, dqs, dks, dvs), lse in zip(_parts(c, q, k, v, o, s["do"], dq, dk, dv), lses):
        hide = ~_seen(c["mask"], c["left"], qs.shape[0], qs.shape[0], qs.device)
        for h in range(c["hkv"]):
            at = slice(h * group, (h + 1) * group)
            qh, dh, kh, vh = qs[:, at], ds[:, at].to(F32), ks[:, h], vs[:, h]
            delta = (dh * os[:, at]).sum(-1).T[..., None]
            p = torch.einsum("qgd,kd->gqk", qh, kh).mul_(scale).sub_(lse[at][..., None]).exp_().masked_fill_(hide, 0.0)
            dvs[:, h] = torch.einsum("gqk,qgd->kd", p, dh).to(dt)
            dp = torch.einsum("qgd,kd->gqk", dh, vh)
            p.mul_(dp.sub_(delta)).mul_(scale)
            dqs[:, at] = torch.einsum("gqk,kd->qgd", p, kh).to(dt)
            dks[:, h] = torch.einsum("gqk,qgd->kd", p, qh).to(dt)
    return [dq, dk, dv]


def _request_scores(s, c, b, cu, n, dtype):
    """[kv heads, heads of a group, new tokens, keys]: request b's scaled scores, -inf where masked."""
    page, hkv = c["page"], c["hkv"]
    ids = s["block_table"][b, : _pages(n, page)].to(I64)
    e = (s["k_exp"][ids].to(I32) - EXP_BIAS)[:, None, :, None]
    k = torch.ldexp(s["k_cache"][ids].to(dtype), e).flatten(0, 1)[:n]
    q = s["q"][cu[b]:cu[b + 1]].to(dtype).unflatten(1, (hkv, -1))
    sc = torch.einsum("qhgd,khd->hgqk", q, k).mul_(_softmax_scale(c))
    return sc.masked_fill_(~_seen(c["mask"], c["left"], q.shape[0], n, q.device), -math.inf)


def _weighed(s, c, dtype):
    """The weights and positions after a call, in this type."""
    page, cu, new = c["page"], [0], _new(c)
    for n in new:
        cu.append(cu[-1] + n)
    after = [max(a, n) for a, n in zip(_lengths(c["batch"], c["lo"], c["hi"]), new)]
    weight, position = s["weight"].to(dtype), s["position"]
    for b, n in enumerate(after):
        sc = _request_scores(s, c, b, cu, n, dtype)
        lse = s["lse"][:, cu[b]:cu[b + 1]].to(dtype).unflatten(0, (c["hkv"], -1))[..., None]
        got = sc.sub_(lse).exp_().sum((1, 2)).T                                 # [keys, kv heads]
        i = torch.arange(n, device=got.device)
        at = s["block_table"][b, i // page].to(I64), slice(None), i % page
        fresh = (i >= n - new[b]) if c["mask"] != "none" else torch.zeros_like(i, dtype=torch.bool)
        weight[at] = torch.where(fresh[:, None], got, c["decay"] * weight[at] + got)
        where = (i.to(I32) + s["position_offsets"][b])[:, None]
        position[at] = torch.where(fresh[:, None], where, position[at])
    return weight, position


def _plain_weigh(s, c):
    weight, position = _weighed(s, c, F32)
    s["weight"].copy_(weight)
    return {"weight": s["weight"], "position": position}


def _kept(s, c):
    """[batch, kv heads, rows]: whether a cached token stays; also the rows' pages and whether a request evicts."""
    page, table = c["page"], s["block_table"]
    i = torch.arange(table.shape[1] * page, device=table.device)
    at = table[:, i // page].clamp(min=0).to(I64)                               # [batch, rows]
    weight = s["weight"][at, :, i % page].transpose(1, 2)
    position = s["position"][at, :, i % page].transpose(1, 2)
    n = s["seqlens"].to(I64)[:, None, None]
    now = n + s["position_offsets"].to(I64)[:, None, None]
    first = (position < c["sink"]) | (position >= now - c["recent"])
    keep = s["keep"].to(I64)[:, None, None]
    evicts = (keep >= 0) & (n > keep)
    # stable sorts: by weight, then what is protected, then what exists
    order = weight.sort(dim=-1, descending=True, stable=True).indices
    for flag in (first, (i < n).expand_as(first)):
        by = flag.gather(-1, order).to(torch.uint8).sort(dim=-1, descending=True, stable=True).indices
        order = order.gather(-1, by)
    rank = torch.empty_like(order).scatter_(-1, order, i.expand_as(order))
    return (rank < keep) & (i < n) | ~evicts & (i < n), at, evicts[:, 0, 0]


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_evict(s, c):
    page, hkv = c["page"], c["hkv"]
    kept, at, evicts = _kept(s, c)
    i = torch.arange(kept.shape[-1], device=kept.device)
    keep = s["keep"].to(I64)[:, None, None]
    front = (i < keep) & evicts[:, None, None]
    hole_b, hole_h, to = torch.nonzero(front & ~kept, as_tuple=True)
    _, _, frm = torch.nonzero((i >= keep) & evicts[:, None, None] & kept, as_tuple=True)
    dst, src = at[hole_b, to], at[hole_b, frm]
    for n in ("weight", "position"):
        s[n][dst, hole_h, to % page] = s[n][src, hole_h, frm % page]
    for n in ("k", "v"):
        raw, exp = s[n + "_cache"].view(torch.uint8), s[n + "_exp"]
        old = exp.to(I32) - EXP_BIAS
        e = old.flatten().scatter_reduce(0, dst * hkv + hole_h, old[src, hole_h], "amax").view_as(old)
        values = raw[src, frm % page, hole_h].view(torch.float8_e4m3fn).to(F32)
        moved = _e4m3(torch.ldexp(values, (old[src, hole_h] - e[dst, hole_h])[:, None]))
        # rows that stay where they are, of pages whose scale grew
        grown = (e > old)[at].transpose(1, 2)                                   # [batch, kv heads, rows]
        b, h, r = torch.nonzero(front & grown, as_tuple=True)
        p = at[b, r]
        values = raw[p, r % page, h].view(torch.float8_e4m3fn).to(F32)
        raw[p, r % page, h] = _e4m3(torch.ldexp(values, (old[p, h] - e[p, h])[:, None]))
        raw[dst, to % page, hole_h] = moved
        exp.copy_((e + EXP_BIAS).to(torch.uint8))
    # pages behind the ones that are needed go back, in order
    n = s["seqlens"].to(I64)
    after = torch.where(evicts, s["keep"].to(I64), n)
    held, need = (n + page - 1) // page, (after + page - 1) // page
    col = torch.arange(s["block_table"].shape[1], device=n.device)
    back = s["block_table"][(col >= need[:, None]) & (col < held[:, None])]
    s["free_pages"][s["free_count"].to(I64) + torch.arange(back.numel(), device=n.device)] = back
    return {**{x: s[x] for x in ("k_cache", "k_exp", "v_cache", "v_exp", "weight", "position", "free_pages")},
            "seqlens": after.to(I32), "position_offsets": s["position_offsets"] + (n - after).to(I32),
            "free_count": s["free_count"] + back.numel()}


PLAIN = {"checkpoint": _plain_checkpoint, "backward": _plain_backward, "weigh": _plain_weigh, "evict": _plain_evict}


# ------------------------------------------------- the package's entry points

CHECKPOINT = ("q", "k", "v", "o", "q_exp", "k_exp", "v_exp", "o_exp")


def _own_checkpoint(B, s, c):
    return B.checkpoint(s["q"], s["k"], s["v"], s["o"])._asdict()


def _own_backward(B, s, c):
    longest = c["hi"]
    packed = dict(cu_seqlens_q=s["cu_seqlens"], cu_seqlens_k=s["cu_seqlens"], max_seqlen_q=longest,
                  max_seqlen_k=longest) if c["packed"] else {}
    return list(B.attn_backward_checkpoint(
        B.AttnCheckpoint(*(s[n] for n in CHECKPOINT)), s["do"], s["lse"], scale=_softmax_scale(c),
        mask=MASKS[c["mask"]], left=c["left"], right=0 if c["mask"] == "window" else -1,
        deterministic=B.DET_ORDERED, check_status=False, **packed))


def _own_weigh(B, s, c):
    cache = B.KvCache(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    weights = B.KvWeights(s["weight"], s["position"], s["status"])
    B.kv_weigh(s["q"], s["lse"], cache, weights, s["block_table"], s["seqlens"], s["cu_seqlens"],
               scale=_softmax_scale(c), mask=MASKS[c["mask"]], left=c["left"],
               right=0 if c["mask"] == "window" else -1, decay=c["decay"], position_offsets=s["position_offsets"],
               max_seqlen_q=c["new"], max_seqlen_k=s["block_table"].shape[1] * c["page"])
    return {"weight": s["weight"], "position": s["position"]}


def _own_evict(B, s, c):
    cache = B.KvCache(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    weights = B.KvWeights(s["weight"], s["position"], s["status"])
    e = B.kv_evict(cache, weights, s["keep"], s["seqlens"], s["position_offsets"], s["block_table"], s["free_pages"],
                   s["free_count"], sink=c["sink"], recent=c["recent"],
                   max_seqlen_k=s["block_table"].shape[1] * c["page"])
    return {**{x: s[x] for x in ("k_cache", "k_exp", "v_cache", "v_exp", "weight", "position", "free_pages")},
            "seqlens": e.seqlens, "position_offsets": e.position_offsets, "free_count": e.free_count}


OWN = {"checkpoint": _own_checkpoint, "backward": _own_backward, "weigh": _own_weigh, "evict": _own_evict}


def run(state):
    c = state["case"]
    if own:
        from head_attention_backward_gb300 import binding as B
        return OWN[c["op"]](B, state, c)
    return PLAIN[c["op"]](state, c)


# --------------------------------------------------------------------- work

def _pairs(mask, left, lq, lk):
    """Query-key pairs that the mask leaves, and the first key that any query sees."""
    if mask == "none":
        return lq * lk, 0
    off = 0 if mask == "top_left" else lk - lq
    if mask != "window":
        return lq * off + lq * (lq + 1) // 2, 0
    return sum(min(off + i, left) + 1 for i in range(lq)), max(0, off - left)


def work(case):
    c = case
    width = c["dqk"] + c["dv"]
    if c["op"] in ("checkpoint", "backward"):
        size = 4 if c["dtype"] == "fp32" else 2
        values = sum(_lens(c)) * (c["hq"] + c["hkv"]) * width
        held = values * (1 + 1 / GROUP)
        if c["op"] == "checkpoint":
            return {"bytes": values * size + held, "flops": 3 * values}
        pairs = sum(_pairs(c["mask"], c["left"], n, n)[0] for n in _lens(c))
        rows = sum(_lens(c))
        return {"bytes": held + size * rows * (c["hq"] * width + c["hkv"] * width) + 4 * rows * c["hq"],
                "flops": 2 * pairs * c["hq"] * (3 * c["dqk"] + 2 * c["dv"])}
    if c["op"] == "weigh":
        pairs = keys = all_keys = 0
        for a, n in zip(_lengths(c["batch"], c["lo"], c["hi"]), _new(c)):
            a = max(a, n)
            p, first = _pairs(c["mask"], c["left"], n, a)
            pairs, keys, all_keys = pairs + p, keys + a - first, all_keys + a
        touched = keys if c["decay"] == 1.0 else all_keys
        tokens = sum(_new(c))
        fresh = tokens if c["mask"] != "none" else 0
        return {"bytes": keys * c["hkv"] * (c["dqk"] + 1.0 / c["page"]) + (8 * touched + 4 * fresh) * c["hkv"] +
                tokens * c["hq"] * (2 * c["dqk"] + 4), "flops": 2 * pairs * c["hq"] * c["dqk"]}
    total = 0.0
    for n in _lengths(c["batch"], c["lo"], c["hi"]):
        if n > c["keep"]:
            # rows that change place where the kept ones lie anywhere
            moved = c["keep"] * (n - c["keep"]) / n
            total += c["hkv"] * (8 * n + 2 * moved * (width + 8))
    return {"bytes": total + 16 * c["batch"], "flops": 0}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    c = case
    if c["op"] == "checkpoint":
        return None                                  # whole numbers: equal or wrong
    s = prepare(case, seed)
    if c["op"] == "backward":
        return _exact_backward(s, c)
    return _exact_weigh(s, c) if c["op"] == "weigh" else _exact_evict(s, c)


def _exact_backward(s, c):
    top = torch.finfo(s["do"].dtype).max
    full = {}
    for n in ("q", "k", "v", "o"):
        step = torch.exp2(s[n + "_exp"].to(F64) - EXP_BIAS).repeat_interleave(GROUP, -1)
        full[n] = (s[n].to(F64) * step).clamp(-top, top)
    grads = {n: torch.zeros_like(full[n]) for n in ("q", "k", "v")}
    scale, group, dev = c["dqk"] ** -0.5, c["hq"] // c["hkv"], s["do"].device
    at = 0
    for b, n in enumerate(_lens(c)):
        pick = (lambda x: x[at:at + n]) if c["packed"] else (lambda x: x[b])
        i, j = torch.arange(n, device=dev)[:, None], torch.arange(n, device=dev)
        hide = torch.zeros((n, n), dtype=torch.bool, device=dev)
        if c["mask"] != "none":                      # equal lengths: both causal corners are the same
            hide = hide | (j > i)
        if c["mask"] == "window":
            hide = hide | (i - j > c["left"])
        lse = (s["lse"][:, at:at + n] if c["packed"] else s["lse"][b]).to(F64)
        for h in range(c["hq"]):
            kv = h // group
            qh, kh, vh = pick(full["q"])[:, h], pick(full["k"])[:, kv], pick(full["v"])[:, kv]
            dh = pick(s["do"])[:, h].to(F64)
            p = torch.exp(qh @ kh.T * scale - lse[h][:, None]).masked_fill(hide, 0.0)
            pick(grads["v"])[:, kv] += p.T @ dh
            ds = p * (dh @ vh.T - (dh * pick(full["o"])[:, h]).sum(-1, keepdim=True)) * scale
            pick(grads["q"])[:, h] = ds @ kh
            pick(grads["k"])[:, kv] += ds.T @ qh
        at += n
    return [grads["q"], grads["k"], grads["v"]]


def _exact_weigh(s, c):
    weight, page = s["weight"].to(F64), c["page"]
    group, at = c["hq"] // c["hkv"], 0
    for b, n in enumerate(s["seqlens"].tolist()):
        lq = _new(c)[b]
        ids = s["block_table"][b, : _pages(n, page)].to(I64)
        j = torch.arange(n, device=ids.device)
        i = torch.arange(n - lq, n, device=ids.device)[:, None]
        hide = torch.zeros((lq, n), dtype=torch.bool, device=ids.device)
        if c["mask"] != "none":
            hide = hide | (j > i)
        if c["mask"] == "window":
            hide = hide | (i - j > c["left"])
        for h in range(c["hkv"]):
            k = (s["k_cache"][ids, :, h].to(F64) *
                 torch.exp2(s["k_exp"][ids, h].to(F64) - EXP_BIAS)[:, None, None]).flatten(0, 1)[:n]
            got = torch.zeros(n, dtype=F64, device=ids.device)
            for x in range(h * group, (h + 1) * group):
                sc = s["q"][at:at + lq, x].to(F64) @ k.T * c["dqk"] ** -0.5
                got += torch.exp(sc - s["lse"][x, at:at + lq].to(F64)[:, None]).masked_fill(hide, 0.0).sum(0)
            before = weight[ids[j // page], h, j % page] * c["decay"]
            if c["mask"] != "none":
                before[n - lq:] = 0.0
            weight[ids[j // page], h, j % page] = before + got
        at += lq
    return {"weight": weight, "position": None}


def _nearest_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, in 64 bits."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _exact_evict(s, c):
    page, keep = c["page"], c["keep"]
    out = {n: s[n].to(F64) for n in ("k_cache", "v_cache", "weight")}
    for b, n in enumerate(s["seqlens"].tolist()):
        if n <= keep:
            continue
        ids = s["block_table"][b, : _pages(n, page)].to(I64)
        j = torch.arange(n, device=ids.device)
        for h in range(c["hkv"]):
            w = s["weight"][ids[j // page], h, j % page].to(F64)
            pos = s["position"][ids[j // page], h, j % page].to(I64)
            now = n + int(c["past"])
            w = torch.where((pos < c["sink"]) | (pos >= now - c["recent"]), torch.full_like(w, math.inf), w)
            stay = torch.zeros(n, dtype=torch.bool, device=ids.device)
            stay[w.sort(descending=True, stable=True).indices[:keep]] = True
            to, frm = j[:keep][~stay[:keep]], j[keep:][stay[keep:]]
            out["weight"][ids[to // page], h, to % page] = s["weight"][ids[frm // page], h, frm % page].to(F64)
            for x in ("k", "v"):
                e = s[x + "_exp"][:, h].to(F64) - EXP_BIAS
                grown = e.clone()
                grown.scatter_reduce_(0, ids[to // page], e[ids[frm // page]], "amax")
                value = out[x + "_cache"]
                moved = value[ids[frm // page], frm % page, h] * torch.exp2(e[ids[frm // page]] -
                                                                            grown[ids[to // page]])[:, None]
                front = j[:keep]
                there = ids[front // page]
                value[there, front % page, h] = _nearest_e4m3(value[there, front % page, h] *
                                                              torch.exp2(e[there] - grown[there])[:, None])
                value[ids[to // page], to % page, h] = _nearest_e4m3(moved)
    return {**{n: None for n in ("k_exp", "v_exp", "position", "free_pages", "seqlens", "position_offsets",
                                 "free_count")}, **out}
