"""The serving operators next to the attention kernels, with their plain forms.

Four operators, used in this order by one serving step (and the first one, in
both directions, by a training step around attn_forward / attn_backward):

* rope: rotary positions with up to four axes, applied to q and k in one call;
  the inverse rotation is its gradient;
* kv_plan: block tables, positions and a slot map from request lengths;
* kv_append: new keys and values quantised to e4m3 into a paged cache with one
  power-of-two scale per page and kv head;
* attn_kv_forward: attention of new tokens over that cache.

`listed()` names the measured cases, `draw()` gives more of the same ranges.
`run(state)` makes one pass: with `own` false in elementary torch operations in
32 bits (angles in 64), with `own` true through this package's entry points.
`exact(case, seed)` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

F64, F32, I32, I64 = torch.float64, torch.float32, torch.int32, torch.int64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MASKS = {"none": 0, "causal": 2, "window": 3}      # attn_mask_t: none, bottom-right causal, window
EXP_BIAS, EXP_MIN, EXP_MAX = 127, -30, 30          # scale of a page and head: 2^(byte - 127)
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the new tokens of a decode batch: the smallest call, all latency
        dict(name="rope_decode", op="rope", rows=64, hq=32, hkv=8, d=128, rot=128, axes=3, dtype="bf16",
             interleaved=False, inverse=False, far=131072),
        # gradients of q and k of a training batch rotated back: half the head rotated, adjacent pairs
        dict(name="rope_gradient", op="rope", rows=2 * 4099, hq=16, hkv=16, d=64, rot=32, axes=2, dtype="fp16",
             interleaved=True, inverse=True, far=4099),
        # packed training tokens or a prompt, time / height / width positions
        dict(name="rope_prompt", op="rope", rows=16384, hq=32, hkv=8, d=128, rot=128, axes=3, dtype="bf16",
             interleaved=False, inverse=False, far=16384),
        # bookkeeping of one decode step
        dict(name="plan_decode", op="plan", batch=64, page=16, lo=100, hi=8192, new=1, prompts=0, prompt=1, leave=0),
        # a busy step: decoding requests, new prompts and requests that leave
        dict(name="plan_mixed", op="plan", batch=500, page=16, lo=1, hi=4096, new=1, prompts=9, prompt=1801, leave=7),
        # one token for each of 64 requests: most pages are partly filled
        dict(name="append_decode", op="append", batch=64, page=16, lo=100, hi=2048, new=1, hkv=8, dqk=128, dv=128,
             dtype="bf16"),
        # ragged prompt pieces behind cached tokens, unequal head dims
        dict(name="append_ragged", op="append", batch=7, page=32, lo=0, hi=700, new=333, hkv=4, dqk=192, dv=128,
             dtype="fp16"),
        # prompts of 16384 tokens in all
        dict(name="append_prompt", op="append", batch=15, page=64, lo=0, hi=0, new=1092, hkv=8, dqk=128, dv=128,
             dtype="bf16"),
        # a small chat batch: latency
        dict(name="attend_small", op="attend", batch=4, page=16, lo=700, hi=1025, new=1, hq=32, hkv=8, dqk=128, dv=128,
             mask="causal", left=-1, dtype="bf16"),
        # a full decode batch of ragged contexts: cache bandwidth
        dict(name="attend_batch", op="attend", batch=64, page=16, lo=500, hi=8192, new=1, hq=32, hkv=8, dqk=128,
             dv=128, mask="causal", left=-1, dtype="bf16"),
        # one request with a very long context
        dict(name="attend_long", op="attend", batch=1, page=64, lo=131072, hi=131072, new=1, hq=32, hkv=8, dqk=128,
             dv=128, mask="causal", left=-1, dtype="fp16"),
        # prompt pieces behind a cached prefix: compute
        dict(name="attend_prompt", op="attend", batch=4, page=16, lo=3500, hi=5120, new=1024, hq=32, hkv=8, dqk=128,
             dv=128, mask="causal", left=-1, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "plan", "append", "attend"))
    if op == "rope":
        d = rng.choice((64, 128, 192, 256))
        return dict(op=op, rows=_spread(rng, 1, 8192), hq=rng.choice((1, 4, 8, 16, 24)), hkv=rng.choice((1, 2, 5, 8)),
                    d=d, rot=rng.choice((d, d // 2, d - 6)), axes=rng.randint(1, 4),
                    dtype=rng.choice(("bf16", "fp16", "fp32")), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, far=_spread(rng, 16, 1 << 20))
    if op == "plan":
        batch = _spread(rng, 1, 1000)
        return dict(op=op, batch=batch, page=rng.choice((16, 32, 64, 128)), lo=rng.randint(0, 50),
                    hi=_spread(rng, 60, 4000), new=rng.randint(0, 3), prompts=rng.randint(0, min(5, batch)),
                    prompt=_spread(rng, 1, 3000), leave=rng.randint(0, batch // 4))
    dqk, dv = rng.choice(((64, 64), (128, 128), (192, 128), (256, 256)))
    page = rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "append":
        batch = _spread(rng, 1, 100)
        lo = rng.randint(0, 300)
        return dict(op=op, batch=batch, page=page, lo=lo, hi=lo + rng.randint(0, 500),
                    new=_spread(rng, 1, max(2, 8000 // batch)), hkv=rng.choice((1, 2, 3, 8)), dqk=dqk, dv=dv,
                    dtype=dtype)
    batch = _spread(rng, 1, 64)
    new = 1 if rng.random() < 0.5 else _spread(rng, 2, max(3, 1000 // batch))
    hi = _spread(rng, new + 1, max(new + 2, min(16384, 131072 // batch)))
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
    mask = rng.choice(("none", "causal", "window"))
    return dict(op=op, batch=batch, page=page, lo=rng.randint(0, hi), hi=hi, new=new, hq=hkv * group, hkv=hkv, dqk=dqk,
                dv=dv, mask=mask, left=_spread(rng, 1, hi) if mask == "window" else -1, dtype=dtype)


def _lengths(n, lo, hi):
    """n lengths of [lo, hi] that depend on nothing but these numbers, hi among them."""
    return [hi if i == 0 else lo + (i * 7919 + 13 * n) % (hi - lo + 1) for i in range(n)]


def _new(c):
    """New tokens of every request (-1: the request leaves)."""
    n = c["batch"]
    if c["op"] != "plan":
        return [c["new"] if i % 3 != 1 else max(1, c["new"] - (i * 31) % c["new"]) for i in range(n)]
    new = [c["prompt"] if i < c["prompts"] else c["new"] for i in range(n)]
    for i in range(c["leave"]):
        new[n - 1 - i] = -1
    return new


def _before(c):
    """Cached tokens of every request before the call."""
    before = _lengths(c["batch"], c["lo"], c["hi"])
    return [0 if i < c.get("prompts", 0) else x for i, x in enumerate(before)]


def _pages(tokens, page):
    return (tokens + page - 1) // page


# ------------------------------------------------------------------ inputs

def _table(lens, page, spare, g, dev):
    """Block table of requests with these lengths, its pages in random order, and the pool's size."""
    need = [_pages(x, page) for x in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g, device=dev).to(I32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=I32, device=dev)
    at = torch.arange(table.shape[1], device=dev)
    n = torch.tensor(need, device=dev)
    table[at < n[:, None]] = order[: sum(need)]
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
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev).to(dt)   # noqa: E731
    s = {"case": c}
    if c["op"] == "rope":
        half = c["rot"] // 2
        s["q"], s["k"] = rand(c["rows"], c["hq"], c["d"]), rand(c["rows"], c["hkv"], c["d"])
        s["positions"] = torch.randint(0, c["far"], (c["axes"], c["rows"]), generator=g, device=dev, dtype=I32)
        # one ladder of frequencies over the pairs, its pairs dealt to the axes in runs
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=F64) / half)
        s["pair_axis"] = (torch.arange(half) * c["axes"] // half).to(torch.uint8)
        s["inv_freq_dev"], s["pair_axis_dev"] = s["inv_freq"].to(dev), s["pair_axis"].to(dev, I64)
        return s
    before, new, page = _before(c), _new(c), c["page"]
    after = [0 if n < 0 else b + n for b, n in zip(before, new)]
    if c["op"] == "plan":
        table, order, pool = _table(before, page, sum(_pages(x, page) for x in after) + 5, g, dev)
        wide = max(_pages(x, page) for x in after + before) + 3
        s["block_table"] = torch.full((c["batch"], wide), -1, dtype=I32, device=dev)
        s["block_table"][:, : table.shape[1]] = table
        used = sum(_pages(x, page) for x in before)
        s["free_pages"] = torch.zeros(pool, dtype=I32, device=dev)
        s["free_pages"][: pool - used] = order[used:]
        s["free_count"] = torch.tensor([pool - used], dtype=I32, device=dev)
        s["seqlens"] = torch.tensor(before, dtype=I32, device=dev)
        s["new_lens"] = torch.tensor(new, dtype=I32, device=dev)
        s["max_tokens"] = max(1, sum(max(n, 0) for n in new) + 16)
        return s
    table, _, pool = _table(after, page, 3, g, dev)
    s["k_cache"], s["k_exp"] = _cache(pool, page, c["hkv"], c["dqk"], g, dev)
    s["v_cache"], s["v_exp"] = _cache(pool, page, c["hkv"], c["dv"], g, dev)
    total = sum(new)
    cu = torch.tensor([0] + new, dtype=I64).cumsum(0)
    if c["op"] == "append":
        b = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(new))
        pos = torch.arange(total) - cu[b] + torch.tensor(before)[b]
        b, pos = b.to(dev), pos.to(dev)
        s["slots"] = table[b, pos // page].to(I64) * page + pos % page
        s["k"], s["v"] = rand(total, c["hkv"], c["dqk"]), rand(total, c["hkv"], c["dv"])
        return s
    s["q"] = rand(total, c["hq"], c["dqk"])
    s["block_table"], s["seqlens"] = table, torch.tensor(after, dtype=I32, device=dev)
    s["cu_seqlens"] = cu.to(dev, I32)
    return s


# ------------------------------------------------------------- plain forms

def _pairs(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])


def _rotated(x, cos, sin, rot, interleaved):
    x = x.to(cos.dtype)
    a, b = _pairs(x, rot, interleaved)
    y = x.clone()
    ya, yb = _pairs(y, rot, interleaved)
    ya.copy_(a * cos - b * sin)
    yb.copy_(b * cos + a * sin)
    return y


def _plain_rope(s, c):
    angle = s["positions"].to(F64)[s["pair_axis_dev"]].T * s["inv_freq_dev"]   # angles of far positions need 64 bits
    cos, sin = angle.cos().to(F32)[:, None], angle.sin().to(F32)[:, None]
    sin = -sin if c["inverse"] else sin
    return [_rotated(s[n], cos, sin, c["rot"], c["interleaved"]).to(s[n].dtype) for n in ("q", "k")]


def _plain_plan(s, c):
    page, table, free = c["page"], s["block_table"], s["free_pages"]
    leaves = s["new_lens"] < 0
    new = s["new_lens"].clamp(min=0)
    held = (s["seqlens"] + page - 1) // page
    at = torch.arange(table.shape[1], device=table.device, dtype=I32)
    # pages of the requests that leave go on top of the stack, in order
    back = torch.where(leaves, held, torch.zeros_like(held))
    back_at = back.cumsum(0) - back
    give = at < back[:, None]
    free[(s["free_count"] + back_at[:, None] + at)[give]] = table[give]
    top = s["free_count"] + back.sum()
    # new pages come off its top
    before = torch.where(leaves, torch.zeros_like(new), s["seqlens"])
    after = before + new
    first = (before + page - 1) // page
    take_n = (after + page - 1) // page - first
    take_at = take_n.cumsum(0) - take_n
    take = (at >= first[:, None]) & (at < (first + take_n)[:, None])
    table[take] = free[(top - 1 - take_at[:, None] - (at - first[:, None]))[take]]
    cu = torch.zeros(new.numel() + 1, dtype=I32, device=new.device)
    cu[1:] = new.cumsum(0)
    t = torch.arange(s["max_tokens"], device=new.device, dtype=I32)
    b = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=new.numel() - 1)
    live = t < cu[-1]
    pos = torch.where(live, before[b] + t - cu[b], torch.zeros_like(t))
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].to(I64) * page + pos % page
    return {"cu_seqlens": cu, "seqlens": after.to(I32), "positions": pos.to(I32),
            "slots": torch.where(live, slot, torch.full_like(slot, -1)),
            "free_count": (top - take_n.sum()).to(I32), "block_table": table, "free_pages": free}


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within the format's range."""
    m, k = torch.frexp(amax)                       # amax = m 2^k, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = k - 9 + (m > 0.875).to(k.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append(s, c):
    page, slots = c["page"], s["slots"]
    pool = s["k_cache"].shape[0]
    at, row = slots // page, slots % page
    # rows in front of a page's first new token are live
    kept = torch.full((pool,), page, dtype=I64, device=slots.device).scatter_reduce(0, at, row, "amin")
    touched = torch.unique(at)
    old_rows = torch.arange(page, device=slots.device) < kept[touched][:, None]
    for x, cache, exp in ((s["k"], s["k_cache"], s["k_exp"]), (s["v"], s["v_cache"], s["v_exp"])):
        x = x.to(F32)
        amax = torch.zeros((pool, x.shape[1]), device=x.device)
        amax.scatter_reduce_(0, at[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        e = _exponent(amax[touched])
        old = exp[touched].to(I32) - EXP_BIAS
        e = torch.where((kept[touched] > 0)[:, None], torch.maximum(old, e), e)
        exp[touched] = (e + EXP_BIAS).to(torch.uint8)
        was = cache[touched].to(F32)
        now = _e4m3(torch.ldexp(was, (old - e)[:, None, :, None])).view(torch.uint8)
        raw = cache.view(torch.uint8)
        raw[touched] = torch.where(old_rows[:, :, None, None], now, raw[touched])
        here = exp[at].to(I32) - EXP_BIAS
        raw[at, row] = _e4m3(torch.ldexp(x, -here[:, :, None])).view(torch.uint8)
    return {n: s[n] for n in ("k_cache", "k_exp", "v_cache", "v_exp")}


def _visible(c, new, after, rows, keys):
    """[batch, rows, keys]: which key of its request each new token sees."""
    dev = after.device
    i = torch.arange(rows, device=dev)[None, :, None] + (after - new)[:, None, None]
    j = torch.arange(keys, device=dev)[None, None, :]
    see = (j < after[:, None, None]).expand(-1, rows, -1)
    if c["mask"] != "none":
        see = see & (j <= i)
    if c["mask"] == "window":
        see = see & (j >= i - c["left"])
    return see


def _softmax_scale(c):
    return 1.0 / math.sqrt(c["dqk"])


def _plain_attend(s, c):
    page, table, q = c["page"], s["block_table"], s["q"]
    batch, hkv = c["batch"], c["hkv"]
    new = s["cu_seqlens"].diff()
    rows, keys = max(_new(c)), table.shape[1] * page
    b = torch.repeat_interleave(torch.arange(batch, device=q.device), new, output_size=q.shape[0])
    i = torch.arange(q.shape[0], device=q.device) - s["cu_seqlens"][b]
    wide = torch.zeros((batch, rows, hkv, c["hq"] // hkv, c["dqk"]), dtype=F32, device=q.device)
    wide[b, i] = q.to(F32).view(q.shape[0], hkv, -1, c["dqk"])
    at = table.clamp(min=0)
    see = _visible(c, new, s["seqlens"], rows, keys)

    def real(cache, exp):   # the values that the bytes stand for: [batch, keys, hkv, d]
        x = torch.ldexp(cache.view(torch.uint8)[at].view(cache.dtype).to(F32),
                        (exp[at].to(I32) - EXP_BIAS)[:, :, None, :, None])
        return x.view(batch, keys, hkv, -1)

    sc = torch.einsum("bqhgd,bkhd->bhgqk", wide, real(s["k_cache"], s["k_exp"])).mul_(_softmax_scale(c))
    sc.masked_fill_(~see[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True)
    v = real(s["v_cache"], s["v_exp"]) * (torch.arange(keys, device=q.device) < s["seqlens"][:, None])[:, :, None, None]
    o = torch.einsum("bhgqk,bkhd->bhgqd", p, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log())[..., 0].flatten(1, 2)                      # [batch, hq, rows]; -inf where nothing is seen
    o = o.flatten(1, 2).transpose(1, 2)                            # [batch, rows, hq, dv]
    return {"o": o[b, i].to(q.dtype), "lse": lse.transpose(1, 2)[b, i].T.contiguous()}


PLAIN = {"rope": _plain_rope, "plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}


# ------------------------------------------------- the package's entry points

def _own_rope(B, s, c):
    return list(B.rope(s["q"], s["k"], s["positions"], s["inv_freq"], pair_axis=s["pair_axis"],
                       interleaved=c["interleaved"], inverse=c["inverse"]))


def _own_plan(B, s, c):
    p = B.kv_plan(s["new_lens"], s["seqlens"], s["block_table"], s["free_pages"], s["free_count"],
                  page_size=c["page"], max_tokens=s["max_tokens"])
    return {"cu_seqlens": p.cu_seqlens, "seqlens": p.seqlens, "positions": p.positions, "slots": p.slots,
            "free_count": p.free_count, "block_table": s["block_table"], "free_pages": s["free_pages"]}


def _own_append(B, s, c):
    cache = B.KvCache(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    B.kv_append(s["k"], s["v"], s["slots"], cache)
    return {n: s[n] for n in ("k_cache", "k_exp", "v_cache", "v_exp")}


def _own_attend(B, s, c):
    cache = B.KvCache(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    o, lse = B.attn_kv_forward(s["q"], cache, s["block_table"], s["seqlens"], s["cu_seqlens"],
                               scale=_softmax_scale(c), mask=MASKS[c["mask"]], left=c["left"],
                               right=0 if c["mask"] == "window" else -1, max_seqlen_q=max(_new(c)),
                               max_seqlen_k=s["block_table"].shape[1] * c["page"])
    return {"o": o, "lse": lse}


OWN = {"rope": _own_rope, "plan": _own_plan, "append": _own_append, "attend": _own_attend}


def run(state):
    c = state["case"]
    if own:
        from head_attention_backward_gb300 import binding as B
        return OWN[c["op"]](B, state, c)
    return PLAIN[c["op"]](state, c)


# --------------------------------------------------------------------- work

def work(case):
    c = case
    size = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "rope":
        values = c["rows"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 2 * values * size + 4 * c["axes"] * c["rows"],
                "flops": 6 * c["rows"] * (c["hq"] + c["hkv"]) * (c["rot"] // 2)}
    before, new, page = _before(c), _new(c), c["page"]
    tokens = sum(max(n, 0) for n in new)
    if c["op"] == "plan":
        back = sum(_pages(b, page) for b, n in zip(before, new) if n < 0)
        take = sum(_pages(b + n, page) - _pages(b, page) for b, n in zip(before, new) if n >= 0)
        return {"bytes": 4 * (4 * c["batch"] + 1) + 8 * (back + take) + 12 * (tokens + 16), "flops": 0}
    width = c["dqk"] + c["dv"]
    if c["op"] == "append":
        touched = sum(_pages(b + n, page) - b // page for b, n in zip(before, new))
        return {"bytes": tokens * (8 + c["hkv"] * width * (size + 1)) + 4 * touched * c["hkv"],
                "flops": 2 * tokens * c["hkv"] * width}
    pairs = cached = 0
    for b, n in zip(before, new):
        first = 0
        if c["mask"] == "none":
            pairs += n * (b + n)
        elif c["mask"] == "causal":
            pairs += n * b + n * (n + 1) // 2
        else:
            pairs += sum(min(b + i, c["left"]) + 1 for i in range(n))
            first = max(0, b - c["left"])
        cached += b + n - first
    return {"bytes": cached * c["hkv"] * (width + 2.0 / page) + tokens * c["hq"] * (width * size + 4),
            "flops": 2 * pairs * c["hq"] * width}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return None                                  # whole numbers: equal or wrong
    if c["op"] == "rope":
        ph = s["positions"].to(F64)[s["pair_axis_dev"].cpu().numpy().tolist()].T * s["inv_freq_dev"]
        turn = torch.polar(torch.ones_like(ph), -ph if c["inverse"] else ph)[:, None]
        out = []
        for x in (s["q"].to(F64), s["k"].to(F64)):
            y, r = x.clone(), c["rot"]
            if c["interleaved"]:
                z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
                y[..., :r] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., : r // 2].contiguous(), x[..., r // 2: r].contiguous()) * turn
                y[..., :r] = torch.cat((z.real, z.imag), -1)
            out.append(y)
        return out
    return _exact_append(s, c) if c["op"] == "append" else _exact_attend(s, c)


def _nearest_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, in 64 bits."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _exact_append(s, c):
    page, out = c["page"], {"k_exp": None, "v_exp": None}
    at, row = (s["slots"] // page), (s["slots"] % page)
    pages, which = torch.unique(at, return_inverse=True)
    first = torch.stack([row[which == i].min() for i in range(len(pages))])
    for n in ("k", "v"):
        x, exp = s[n].to(F64), s[n + "_exp"].to(F64) - EXP_BIAS
        value = s[n + "_cache"].to(F64)
        top = torch.stack([x[which == i].abs().amax(-1).amax(0) for i in range(len(pages))])     # [pages, hkv]
        e = torch.where(top > 0, torch.ceil(torch.log2(top / E4M3_MAX)), torch.full_like(top, EXP_MIN))
        e = e.clamp(EXP_MIN, EXP_MAX)
        e = torch.where((first > 0)[:, None], torch.maximum(e, exp[pages]), e)
        held = _nearest_e4m3(value[pages] * torch.exp2(exp[pages] - e)[:, None, :, None])
        live = torch.arange(page, device=x.device) < first[:, None]
        value[pages] = torch.where(live[:, :, None, None], held, value[pages])
        value[at, row] = _nearest_e4m3(x * torch.exp2(-e[which])[:, :, None])
        out[n + "_cache"] = value
    return out


def _exact_attend(s, c):
    page, q = c["page"], s["q"].to(F64)
    group = c["hq"] // c["hkv"]
    o = torch.zeros(q.shape[0], c["hq"], c["dv"], dtype=F64, device=q.device)
    lse = torch.full((c["hq"], q.shape[0]), -math.inf, dtype=F64, device=q.device)
    cu = s["cu_seqlens"].tolist()
    for b, n in enumerate(s["seqlens"].tolist()):
        lo, hi = cu[b], cu[b + 1]
        if n == 0 or hi == lo:
            continue
        ids = s["block_table"][b, : _pages(n, page)].to(I64)
        k = (s["k_cache"][ids].to(F64) * torch.exp2(s["k_exp"][ids].to(F64) - EXP_BIAS)[:, None, :, None]).flatten(0, 1)
        v = (s["v_cache"][ids].to(F64) * torch.exp2(s["v_exp"][ids].to(F64) - EXP_BIAS)[:, None, :, None]).flatten(0, 1)
        i = torch.arange(n - (hi - lo), n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)
        hide = torch.zeros(hi - lo, n, dtype=torch.bool, device=q.device)
        if c["mask"] != "none":
            hide = hide | (j > i)
        if c["mask"] == "window":
            hide = hide | (j < i - c["left"])
        for h in range(c["hkv"]):
            qs = q[lo:hi, h * group:(h + 1) * group].transpose(0, 1)                            # [group, rows, dqk]
            sc = (qs @ k[:n, h].T * _softmax_scale(c)).masked_fill(hide, -math.inf)
            part = torch.logsumexp(sc, -1)
            w = torch.exp(sc - torch.where(part == -math.inf, torch.zeros_like(part), part)[..., None])
            o[lo:hi, h * group:(h + 1) * group] = (w @ v[:n, h]).transpose(0, 1)
            lse[h * group:(h + 1) * group, lo:hi] = part
    return {"o": o, "lse": lse}
