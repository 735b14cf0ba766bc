"""The paged 8-bit cache on the GPU: bookkeeping, append and attention against
the fp64 oracle, alone and as the serving step they make up."""
import math

import pytest
import torch

from oracle import kv_ref
from tests.kv_cases import block_table, check_attend, random_cache
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

I32 = torch.int32
DIMS = [(64, 64), (128, 128), (192, 128), (256, 256)]


def dev(x, dtype=I32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def handle(B, kc, vc, ke, ve):
    f8 = torch.float8_e4m3fn
    return B.KvCache(kc.cuda().view(f8), vc.cuda().view(f8), ke.cuda(), ve.cuda())


# ---------------------------------------------------------------------- plan

PLANS = [
    # page, new_lens, seqlens, extra free pages, extra token capacity
    (16, [1], [0], 0, 0),
    (16, [0], [0], 1, 3),
    (16, [1, 1, 1], [15, 16, 17], 0, 0),
    (32, [0, 5, -1, 100, 1, -1, 0], [0, 0, 70, 3, 32, 0, 64], 0, 7),
    (64, [-1, -1], [64, 1], 0, 0),
    (16, [-1, 40], [33, 0], -2, 1),          # the new request needs the pages given back
    (256, [1000, 1], [1000, 255], 5, 0),
    (16, [7000, 3, 1], [0, 10, 5000], 3, 11),
]


@pytest.mark.parametrize("page,new,lens,spare,more", PLANS)
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(B, page, new, lens, spare, more, in_place):
    g = torch.Generator().manual_seed(len(new))
    held = [(n + page - 1) // page for n in lens]
    grown = [(max(0, n) + (0 if n < 0 else x) + page - 1) // page for n, x in zip(new, lens)]
    need = sum(max(0, a - h) for a, h in zip(grown, held))
    pool = sum(held) + need + max(spare, 0)
    order = torch.randperm(pool, generator=g).tolist()
    cols = max(grown + held) + 2
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-1] * (cols - h))
        at += h
    free = order[at:]
    if spare < 0:
        free = free[:spare]
    count = len(free)
    free = free + [-7] * (pool - count)
    cap = sum(max(n, 0) for n in new) + more
    td = dev(table)
    wide = torch.full((len(new), cols + 5), -3, dtype=I32, device="cuda")   # rows further apart than they are long
    wide[:, :cols] = td
    td = wide[:, :cols]
    fd, nd, ld, cd = dev(free), dev(new), dev(lens), dev([count])
    out = None
    if in_place:
        out = B.KvPlan(torch.empty(len(new) + 1, dtype=I32, device="cuda"), ld, torch.empty(cap, dtype=I32, device="cuda"),
                       torch.empty(cap, dtype=torch.int64, device="cuda"), cd, dev([5]))
    p = B.kv_plan(nd, ld, td, fd, cd, page_size=page, max_tokens=cap, out=out)
    p.check()
    cu, after, pos, slots, left = kv_ref.plan(new, lens, table, free, count, page, cap)
    assert p.cu_seqlens.tolist() == cu and p.seqlens.tolist() == after
    assert p.positions.tolist() == pos and p.slots.tolist() == slots
    assert p.free_count.tolist() == [left] and td.tolist() == table and fd.tolist() == free
    assert bool((wide[:, cols:] == -3).all())
    if not in_place:
        assert ld.tolist() == lens and cd.tolist() == [count]


@pytest.mark.parametrize("batch", [1000, 1025, 8192])
def test_plan_many_requests(B, batch):
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 60, (batch,), generator=g).tolist()
    new = torch.randint(-1, 5, (batch,), generator=g).tolist()
    table, pool = block_table(lens, 16, g, extra_pages=batch, extra_cols=2)
    used = {p for row in table for p in row if p >= 0}
    free = [p for p in range(pool) if p not in used]
    count = len(free)
    free += [0] * (pool - count)
    cap = sum(max(n, 0) for n in new) + 100
    td, fd = dev(table), dev(free)
    p = B.kv_plan(dev(new), dev(lens), td, fd, dev([count]), page_size=16, max_tokens=cap)
    p.check()
    cu, after, pos, slots, left = kv_ref.plan(new, lens, table, free, count, 16, cap)
    assert p.cu_seqlens.tolist() == cu and p.seqlens.tolist() == after
    assert p.positions.tolist() == pos and p.slots.tolist() == slots
    assert p.free_count.tolist() == [left] and td.tolist() == table and fd.tolist() == free


@pytest.mark.parametrize("what,status", [
    ("len below zero", -7), ("len past the table", -7), ("grows past the table", -7), ("new below -1", -7),
    ("too many tokens", -7), ("free_count negative", -7), ("free_count past the pool", -7), ("gives back too many", -7),
    ("out of pages", -9), ("pops a bad page", -8), ("gives back a bad page", -8)])
def test_plan_refused_step_changes_nothing(B, what, status):
    page, cols, pool = 16, 4, 12
    new, lens, count, cap = [3, -1, 20], [10, 33, 0], 8, 40
    table = [[0, -1, -1, -1], [1, 2, 3, -1], [-1, -1, -1, -1]]
    free = [4, 5, 6, 7, 8, 9, 10, 11] + [0] * 4
    if what == "len below zero":
        lens[0] = -1
    elif what == "len past the table":
        lens[1] = page * cols + 1
    elif what == "grows past the table":
        new[2] = page * cols + 1
        cap = 100
    elif what == "new below -1":
        new[2] = -2
    elif what == "too many tokens":
        cap = 22
    elif what == "free_count negative":
        count = -1
    elif what == "free_count past the pool":
        count = pool + 1
    elif what == "gives back too many":
        count = pool - 2
    elif what == "out of pages":
        count, new, cap = 1, [3, 0, 40], 43
    elif what == "pops a bad page":
        free[7], new = pool, [3, 0, 20]
    elif what == "gives back a bad page":
        table[1][1] = -1
    td, fd, ld, cd = dev(table), dev(free), dev(lens), dev([count])
    p = B.kv_plan(dev(new), ld, td, fd, cd, page_size=page, max_tokens=cap)
    assert int(p.status) == status
    with pytest.raises(B.AttnError):
        p.check()
    assert td.tolist() == table and fd.tolist() == free
    assert p.seqlens.tolist() == lens and p.free_count.tolist() == [count]
    assert p.cu_seqlens.tolist() == [0, 0, 0, 0] and p.slots.tolist() == [-1] * cap


def test_plan_refused_step_with_many_tokens(B):
    """The slots of many tokens are written by a kernel of their own: it sees the
    refusal too."""
    cap = 9000
    td, fd = dev([[0, -1], [-1, -1]]), dev([1, 2, 3, 0])
    for new, status in (([1, 33], -7), ([1, 0], 0)):
        p = B.kv_plan(dev(new), dev([3, 0]), td, fd, dev([3]), page_size=16, max_tokens=cap)
        assert int(p.status) == status
        n = 0 if status else 1
        assert p.slots[:n].tolist() == [3] * n and bool((p.slots[n:] == -1).all())
        assert bool((p.positions[n:] == 0).all()) and p.cu_seqlens.tolist() == [0, n, n]


# -------------------------------------------------------------------- append

def runs(spec, page):
    """Slots of (page number, first row, count) runs; None: a skipped token."""
    out = []
    for r in spec:
        out += [-1] if r is None else list(range(r[0] * page + r[1], r[0] * page + r[1] + r[2]))
    return out


@pytest.mark.parametrize("dqk,dv", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,spec", [
    (16, [(3, 0, 1)]),
    (16, [(3, 15, 1), None, (0, 0, 16), (1, 0, 16), (2, 0, 5)]),
    (16, [(i, 5, 1) for i in range(20)] + [None] * 14),
    (32, [(0, 31, 1), (1, 0, 32), (5, 0, 32), (4, 7, 20), None, (2, 3, 1)]),
    (256, [(1, 100, 156), (2, 0, 256), (0, 0, 3)]),
])
def test_append(B, dqk, dv, dtype, page, spec):
    heads, pages = 3, 22
    g = torch.Generator().manual_seed(dqk + page)
    kc, ke = random_cache(pages, page, heads, dqk, g, 12)
    vc, ve = random_cache(pages, page, heads, dv, g, 12)
    slots = runs(spec, page)
    n = len(slots)
    k = torch.randn((n, heads, dqk), generator=g)
    v = torch.randn((n, heads, dv), generator=g)
    k = (k * 2.0 ** torch.randint(-12, 12, (n, 1, 1), generator=g)).to(dtype)
    v = (v * 2.0 ** torch.randint(-3, 3, (n, heads, 1), generator=g)).to(dtype)
    k[n // 2] = 0
    v[0, 0] = 448.0                                   # exactly a scale's largest value
    c = handle(B, kc, vc, ke, ve)
    B.kv_append(k.cuda(), v.cuda(), dev(slots, torch.int64), c)
    kv_ref.append(kc, ke, k, slots)
    kv_ref.append(vc, ve, v, slots)
    for name, got, ref in (("k", c.k, kc), ("v", c.v, vc), ("k_exp", c.k_exp, ke), ("v_exp", c.v_exp, ve)):
        assert torch.equal(got.view(torch.uint8).cpu(), ref), name


def test_append_odd_values(B):
    """Zeros, NaN, infinities, subnormals, magnitudes past the scale range, and
    scale bytes outside the format's range."""
    g = torch.Generator().manual_seed(9)
    kc, ke = random_cache(6, 16, 2, 64, g)
    vc, ve = random_cache(6, 16, 2, 64, g)
    ke[3], ve[3], ke[4] = 255, 0, 180
    slots = runs([(0, 0, 2), (1, 4, 3), (2, 0, 1), (3, 2, 2), (4, 1, 1), (5, 0, 1)], 16)
    n = len(slots)
    k, v = torch.randn((n, 2, 64), generator=g), torch.randn((n, 2, 64), generator=g)
    k[0], k[1] = 0.0, -0.0
    k[2, 0, 5], k[3, 1, 7], v[2, :, :3] = math.nan, math.inf, -math.inf
    k[5] = math.nan
    k[6] *= 1e-38
    v[6] *= 3e38
    v[9] *= 1e-30
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c = handle(B, kc, vc, ke, ve)
    B.kv_append(k.cuda(), v.cuda(), dev(slots, torch.int64), c)
    kv_ref.append(kc, ke, k, slots)
    kv_ref.append(vc, ve, v, slots)
    nan = lambda x: (x & 127) == 127   # noqa: E731
    for got, ref in ((c.k, kc), (c.v, vc)):
        got = got.view(torch.uint8).cpu()
        assert torch.equal(nan(got), nan(ref)) and torch.equal(got[~nan(ref)], ref[~nan(ref)])
    assert torch.equal(c.k_exp.cpu(), ke) and torch.equal(c.v_exp.cpu(), ve)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_runs_out_of_order(B, page):
    """Tokens of several pages interleaved, a page filled backwards, gaps of up
    to page_size - 1 skipped tokens inside a run, a run across CTA tiles."""
    heads, d = 2, 64
    g = torch.Generator().manual_seed(page)
    slots = []
    for i in range(8):                                    # pages 0 and 1 in turn, from rows 3 and 0
        slots += [3 + i, page + i]
    slots += list(range(3 * page - 1, 2 * page - 1, -1))   # page 2 backwards
    for i in range(4):                                    # page 3 from row 2, as far apart as allowed
        slots += [3 * page + 2 + i] + [-1] * (page - 1)
    slots += list(range(4 * page + 1, 5 * page)) + [-1] * 40 + [5 * page + 7, 6 * page, 1 << 40, -5]
    kc, ke = random_cache(7, page, heads, d, g, 10)
    vc, ve = random_cache(7, page, heads, d, g, 10)
    k, v = (torch.randn((len(slots), heads, d), generator=g).to(torch.bfloat16) for _ in range(2))
    c = handle(B, kc, vc, ke, ve)
    B.kv_append(k.cuda(), v.cuda(), dev(slots, torch.int64), c)
    kv_ref.append(kc, ke, k, slots)
    kv_ref.append(vc, ve, v, slots)
    for got, ref in ((c.k, kc), (c.v, vc), (c.k_exp, ke), (c.v_exp, ve)):
        assert torch.equal(got.view(torch.uint8).cpu(), ref)


@pytest.mark.parametrize("tokens", [1, 300, 5000])
def test_append_many_tokens_strided(B, tokens):
    """A long prompt into pages in any order, k and v as slices of a packed
    projection, the cache with its heads outside the rows, some tokens padded."""
    page, heads, d = 64, 2, 128
    g = torch.Generator().manual_seed(tokens)
    pages = (tokens + page - 1) // page + 2
    order = torch.randperm(pages, generator=g).tolist()
    first = 37
    slots = [order[(first + t) // page] * page + (first + t) % page for t in range(tokens)]
    if tokens > 10:
        for t in (3, 4, tokens - 1):
            slots[t] = -1
    kc, ke = random_cache(pages, page, heads, d, g)
    vc, ve = random_cache(pages, page, heads, d, g)
    kv = torch.randn((tokens, 2 * heads + 1, d), generator=g).to(torch.float16)
    kvd = kv.cuda()
    f8 = torch.float8_e4m3fn
    kd, vd = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    c = B.KvCache(kd.view(f8), vd.view(f8), ke.cuda(), ve.cuda())
    B.kv_append(kvd[:, :heads], kvd[:, heads + 1:], dev(slots, torch.int64), c)
    kv_ref.append(kc, ke, kv[:, :heads], slots)
    kv_ref.append(vc, ve, kv[:, heads + 1:], slots)
    for got, ref in ((kd, kc), (vd, vc), (c.k_exp, ke), (c.v_exp, ve)):
        assert torch.equal(got.cpu(), ref)


# -------------------------------------------------------------------- attend

ATTEND = [
    # page, lens (cached incl. new), new, heads (kv, per kv), mask, left, right
    (16, [1], [1], 1, 1, 2, -1, -1),
    (16, [0, 5, 16, 17], [1, 1, 1, 1], 2, 4, 2, -1, -1),
    (32, [100, 0, 33, 700], [1, 0, 1, 1], 2, 1, 0, -1, -1),
    (16, [1000, 257, 64], [1, 1, 1], 1, 16, 3, 100, 0),
    (64, [300, 40], [7, 40], 2, 3, 2, -1, -1),
    (16, [50, 3, 90], [5, 6, 33], 1, 5, 2, -1, -1),          # more queries than keys: rows that see nothing
    (16, [50, 200, 90], [5, 16, 33], 2, 2, 3, 9, 2),
    (16, [80, 70], [9, 4], 1, 2, 3, 0, 0),
    (32, [60, 90], [60, 33], 2, 2, 1, -1, -1),               # top-left
    (128, [500, 129], [3, 17], 1, 8, 0, -1, -1),             # cross attention
    (16, [400, 200], [1, 1], 1, 33, 2, -1, -1),              # more heads in a group than one row tile
    (256, [5000], [1], 2, 8, 2, -1, -1),
    (16, [9000, 100], [1, 2], 1, 4, 2, -1, -1),              # many splits, and one
    (16, [300, 1000, 40, 0, 129], [130, 1, 32, 50, 129], 2, 4, 2, -1, -1),   # long and short segments together
    (32, [700, 33], [200, 33], 1, 2, 3, 150, 3),
    (64, [128, 600], [300, 129], 2, 1, 0, -1, -1),           # cross attention of a prompt
]


def weights(dtype, longest):
    """Type that the softmax weights are rounded to: fp16, and for long segments
    (from 25 tokens on at the earliest: 16-bit products on expanded keys) the
    type of q."""
    return dtype if longest > 24 else torch.float16


def attend_case(dqk, dv, dtype, page, lens, new, hkv, group, seed=0, q_scale=1.0):
    g = torch.Generator().manual_seed(seed + dqk + page)
    table, pool = block_table(lens, page, g)
    kc, ke = random_cache(pool, page, hkv, dqk, g)
    vc, ve = random_cache(pool, page, hkv, dv, g)
    q = (torch.randn((sum(new), hkv * group, dqk), generator=g) * q_scale).to(dtype)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return q, table, kc, vc, ke, ve, cu


@pytest.mark.parametrize("dqk,dv", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,lens,new,hkv,group,mask,left,right", ATTEND)
def test_attend(B, dqk, dv, dtype, page, lens, new, hkv, group, mask, left, right):
    q, table, kc, vc, ke, ve, cu = attend_case(dqk, dv, dtype, page, lens, new, hkv, group)
    scale = dqk ** -0.5
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=scale,
                               mask=mask, left=left, right=right, max_seqlen_q=max(new), max_seqlen_k=max(lens),
                               check_status=True)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, scale, mask, left, right)
    check_attend(o, lse, ref, dtype, dqk, max(lens), weights(dtype, max(new)), what=f"{page} {lens} {new}")


@pytest.mark.parametrize("scale", [-0.1, 3.0, 1e-6])
def test_attend_scales(B, scale):
    """Negative, large (one key takes all) and tiny softmax scales; q rows of
    very different magnitudes, one of them zero."""
    q, table, kc, vc, ke, ve, cu = attend_case(128, 128, torch.bfloat16, 16, [333, 50], [1, 3], 2, 4)
    q = (q.float() * (2.0 ** torch.tensor([-40, 0, 3, -120])).view(4, 1, 1)).to(torch.bfloat16)
    q[1, 3] = 0
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev([333, 50]), dev(cu), scale=scale,
                               max_seqlen_q=3, max_seqlen_k=400, check_status=True)
    ref = kv_ref.attend(q, cu, [333, 50], table, kc, vc, ke, ve, scale, 2)
    check_attend(o, lse, ref, torch.bfloat16, 128, 333)


def test_attend_scale_extremes(B):
    """Pages at both ends of the scale range next to each other, and a page of
    tiny values that takes nearly all the weight."""
    lens, new = [16 * 12], [1]
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.float16, 16, lens, new, 1, 2)
    ve[table[0][3]], ve[table[0][4]], ve[table[0][5]], ve[table[0][9]] = 157, 97, 255, 0
    ke[table[0][4]], ke[table[0][7]] = 127 - 5, 97
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.125,
                               max_seqlen_q=1, max_seqlen_k=192)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.125, 2)
    huge = ref[0].abs() > 65504 * (1 + 2.0 ** -11)
    assert bool(huge.any())                      # fp16 outputs overflow there, as they should
    assert bool(torch.isinf(o.cpu()[huge]).all())
    ve[table[0][3]], ve[table[0][5]] = 127, 120
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.125,
                               max_seqlen_q=1, max_seqlen_k=192)
    check_attend(o, lse, kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.125, 2), torch.float16, 64, 192)


@pytest.mark.parametrize("dqk,dv", DIMS)
def test_attend_ignores_what_it_must_not_see(B, dqk, dv):
    """NaN bytes in cache rows past the length, outside a single token's window
    and in other pages; block-table entries past the length point anywhere."""
    lens, new, page = [37, 100, 64], [1, 1, 1], 32
    q, table, kc, vc, ke, ve, cu = attend_case(dqk, dv, torch.bfloat16, page, lens, new, 2, 2)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.1, 3, 20, 0)
    for b, n in enumerate(lens):
        for j in range(n):
            if j < n - 21:
                kc[table[b][j // page], j % page] = 127
                vc[table[b][j // page], j % page] = 255
        last = table[b][(n - 1) // page]
        if n % page:
            kc[last, n % page:], vc[last, n % page:] = 255, 127
        for j in range((n + page - 1) // page, len(table[b])):
            table[b][j] = 10 ** 9 if j % 2 else -5
    used = {p for b, n in enumerate(lens) for p in table[b][: (n + page - 1) // page]}
    for p in range(kc.shape[0]):
        if p not in used:
            kc[p], vc[p] = 127, 127
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.1, mask=3,
                               left=20, right=0, max_seqlen_q=1, max_seqlen_k=128, check_status=True)
    check_attend(o, lse, ref, torch.bfloat16, dqk, 100)


def test_attend_layouts_and_padding(B):
    """q and o as slices of wider tensors, the cache with heads outside the
    rows, padded segment starts; rows of no segment stay as they were."""
    lens, new, page, hkv, group, d = [90, 30, 200], [2, 5, 1], 16, 2, 4, 128
    q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.bfloat16, page, lens, new, hkv, group)
    starts, total = [3, 6, 20, 25], 25
    wide = torch.randn((total, hkv * group + 3, d), dtype=torch.bfloat16, device="cuda")
    for b in range(3):
        wide[starts[b]:starts[b] + new[b], 1:1 + hkv * group] = q[cu[b]:cu[b + 1]].cuda()
    f8 = torch.float8_e4m3fn
    kd, vd = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2).view(f8) for x in (kc, vc))
    ow = torch.full((total, hkv * group + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hkv * group, total), 5.0, device="cuda")
    B.attn_kv_forward(wide[:, 1:1 + hkv * group], B.KvCache(kd, vd, ke.cuda(), ve.cuda()), dev(table), dev(lens), dev(cu),
                      scale=0.1, max_seqlen_q=5, max_seqlen_k=200, cu_seqlens_q_padded=dev(starts),
                      out=(ow[:, 1:-1], lse), check_status=True)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.1, 2)
    rows = [starts[b] + i for b in range(3) for i in range(new[b])]
    check_attend(ow[rows][:, 1:-1], lse[:, rows], ref, torch.bfloat16, d, 200)
    others = [r for r in range(total) if r not in rows]
    assert bool((ow[others] == 7).all()) and bool((lse[:, others] == 5).all())
    assert bool((ow[:, 0] == 7).all()) and bool((ow[:, -1] == 7).all())


def test_attend_reports_bad_lengths_and_pages(B):
    lens, new, page = [90, 30], [1, 1], 16
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, page, lens, new, 1, 2)
    c, qd = handle(B, kc, vc, ke, ve), q.cuda()
    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=96, check_status=True)
    B.attn_kv_forward(qd, c, dev(table), dev(lens), dev(cu), **kw)
    for bad_cu in ([0, 1, 3], [0, -1, 0], [-1, 0, 1]):
        with pytest.raises(B.AttnError) as e:
            B.attn_kv_forward(qd, c, dev(table), dev(lens), dev(bad_cu), **kw)
        assert e.value.status == B.ATTN_ERR_BAD_SEQLENS
    for bad in ([97, 30], [90, -1], [2 ** 31 - 1, 30]):
        with pytest.raises(B.AttnError) as e:
            B.attn_kv_forward(qd, c, dev(table), dev(bad), dev(cu), **kw)
        assert e.value.status == B.ATTN_ERR_BAD_SEQLENS
    # tokens of a page outside the cache are masked, the other request is untouched
    hole = [list(r) for r in table]
    hole[0][2] = kc.shape[0]
    with pytest.raises(B.AttnError) as e:
        B.attn_kv_forward(qd, c, dev(hole), dev(lens), dev(cu), **kw)
    assert e.value.status == B.ATTN_ERR_BAD_PAGE
    kw["check_status"] = False
    o, lse = B.attn_kv_forward(qd, c, dev(hole), dev(lens), dev(cu), **kw)
    k2, v2 = kc.clone(), vc.clone()
    ref = kv_ref.attend(q, cu, [0, 30], table, k2, v2, ke, ve, 0.1, 2)
    check_attend(o[1:], lse[:, 1:], tuple(x[1:] if i in (0, 2) else x[:, 1:] for i, x in enumerate(ref)),
                 torch.bfloat16, 64, 90)
    # reported wherever it is seen: here only by the last of 40 causal queries
    q2 = q[:1].expand(41, -1, -1).contiguous()
    late = [list(r) for r in table]
    late[0][5] = -1
    with pytest.raises(B.AttnError) as e:
        B.attn_kv_forward(q2.cuda(), c, dev(late), dev([90, 30]), dev([0, 40, 41]), scale=0.1, max_seqlen_q=40,
                          max_seqlen_k=96, check_status=True)
    assert e.value.status == B.ATTN_ERR_BAD_PAGE
    short = [table[0][:2] + table[0][3:], table[1]]
    ref = kv_ref.attend(q, cu, [74, 30], short, kc, vc, ke, ve, 0.1, 2)
    check_attend(o, lse, ref, torch.bfloat16, 64, 90)


def test_attend_long_segments_in_groups(B):
    """Expanded keys that do not fit the workspace's limit at once: max_seqlen_k
    of 2^18 at 8 heads of 128 + 128 columns is 1 GiB for each of three segments.
    A page outside the cache empties the keys of its (long) segment only."""
    lens, new, page, d = [200, 190, 1, 333], [164, 190, 1, 140], 16, 128
    q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.bfloat16, page, lens, new, 8, 1)
    cols = 2 ** 18 // page
    wide = torch.full((4, cols), -1, dtype=I32)
    wide[:, : len(table[0])] = torch.tensor(table, dtype=I32)
    c = handle(B, kc, vc, ke, ve)
    kw = dict(scale=0.1, max_seqlen_q=190, max_seqlen_k=2 ** 18)
    o, lse = B.attn_kv_forward(q.cuda(), c, wide.cuda(), dev(lens), dev(cu), check_status=True, **kw)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.1, 2)
    check_attend(o, lse, ref, torch.bfloat16, d, 333, torch.bfloat16)
    wide[1, 2] = kc.shape[0] + 5
    with pytest.raises(B.AttnError) as e:
        B.attn_kv_forward(q.cuda(), c, wide.cuda(), dev(lens), dev(cu), check_status=True, **kw)
    assert e.value.status == B.ATTN_ERR_BAD_PAGE
    o, lse = B.attn_kv_forward(q.cuda(), c, wide.cuda(), dev(lens), dev(cu), **kw)
    ref = kv_ref.attend(q, cu, [200, 0, 1, 333], table, kc, vc, ke, ve, 0.1, 2)
    check_attend(o, lse, ref, torch.bfloat16, d, 333, torch.bfloat16)


SPLIT = [
    # page, lens, new, heads (kv, per kv), mask, left, right: few query tiles over
    # thousands of keys, so that CTAs share a tile's keys
    (16, [5000], [130], 1, 1, 2, -1, -1),
    (64, [4100, 300, 2200], [64, 130, 1], 1, 3, 2, -1, -1),     # groups that do not divide 128, one tile unsplit
    (32, [3000, 2100], [121, 50], 2, 5, 0, -1, -1),
    (16, [2500, 5000], [90, 600], 1, 2, 3, 1500, 40),           # windows that end inside the splits
    (16, [4000], [200], 1, 4, 1, -1, -1),                       # top-left: one tile of keys
    (128, [2600, 100], [2600, 140], 1, 1, 2, -1, -1),           # from one key tile to all of them
    (16, [3000], [30], 1, 64, 2, -1, -1),
    (16, [2200], [26], 1, 128, 2, -1, -1),                      # one token fills a tile
    (16, [2200], [26], 1, 129, 2, -1, -1),                      # more heads than a tile: never long
]


@pytest.mark.parametrize("dqk,dv,dtype", [(64, 64, torch.float16), (128, 128, torch.bfloat16), (192, 128, torch.bfloat16)])
@pytest.mark.parametrize("page,lens,new,hkv,group,mask,left,right", SPLIT)
def test_attend_long_segments_split(B, dqk, dv, dtype, page, lens, new, hkv, group, mask, left, right):
    """Also the same bits when run again, and NaN in the cache rows that no query
    sees, whose pages are not looked up."""
    q, table, kc, vc, ke, ve, cu = attend_case(dqk, dv, dtype, page, lens, new, hkv, group)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.1, mask, left, right)
    for b, n in enumerate(lens):
        seen = [(max(0, n - new[b] - left), n) if mask == 3 else (0, min(n, new[b])) if mask == 1 else (0, n)][0]
        for i in range((n + page - 1) // page):
            rows = [r for r in range(page) if not seen[0] <= i * page + r < seen[1]]
            if rows:
                kc[table[b][i], rows], vc[table[b][i], rows] = 127, 255
            if len(rows) == page:
                table[b][i] = -7
    args = (q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu))
    kw = dict(scale=0.1, mask=mask, left=left, right=right, max_seqlen_q=max(new), max_seqlen_k=max(lens))
    o, lse = B.attn_kv_forward(*args, check_status=True, **kw)
    check_attend(o, lse, ref, dtype, dqk, max(lens), weights(dtype, max(new)), what=f"{page} {lens} {new}")
    again = B.attn_kv_forward(*args, **kw)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_attend_long_segments_in_a_wide_buffer(B):
    """Split long segments in a q of far more rows than they have: the parts
    follow the segments, not the buffer."""
    lens, new, d, total = [3000, 2600, 40], [60, 130, 3], 64, 40000
    q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.bfloat16, 16, lens, new, 1, 2)
    starts = [39000, 20, 30000, 39900]
    wide, out = (torch.zeros((total, 2, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.full((2, total), 9.0, device="cuda")
    rows = [starts[b] + i for b in range(3) for i in range(new[b])]
    wide[rows] = q.cuda()
    p = B.AttnKvFwdParams(dtype=B.ATTN_BF16, batch=3, nhead_q=2, total_q=total, max_seqlen_q=130, max_seqlen_k=3000,
                          max_blocks=len(table[0]), mask=2, softmax_scale=0.1,
                          cache=B.AttnKvCache(num_pages=400, page_size=16, nhead_kv=1, d_qk=d, d_v=d))
    st, size = B.attn_kv_fwd_workspace_size(p)
    assert st == 0 and size < 32 << 20
    B.attn_kv_forward(wide, handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.1, max_seqlen_q=130,
                      max_seqlen_k=3000, cu_seqlens_q_padded=dev(starts), out=(out, lse), check_status=True,
                      workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.1, 2)
    check_attend(out[rows], lse[:, rows], ref, torch.bfloat16, d, 3000, torch.bfloat16)
    others = torch.ones(total, dtype=torch.bool)
    others[rows] = False
    assert bool((out[others.cuda()] == 0).all()) and bool((lse[:, others.cuda()] == 9).all())


@pytest.mark.parametrize("batch,group,longest,scale", [(70, 4, 7, 0.1), (300, 1, 20, 0.1), (5, 8, 24, 0.1), (1100, 2, 6, 0.1),
                                                       (40, 4, 130, -0.1)])
def test_attend_few_rows_under_a_loose_bound(B, batch, group, longest, scale):
    """max_seqlen_q far above most lengths: the grid follows the rows that q has.
    Empty segments first, last and in between; lengths that go back and more rows
    than q has are reported."""
    g = torch.Generator().manual_seed(batch)
    new = torch.randint(0, 3, (batch,), generator=g).tolist()
    new[0], new[batch // 2], new[-1] = 0, longest, 0
    lens = torch.randint(0, 60, (batch,), generator=g).tolist()
    lens[batch // 2] = 900
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, lens, new, 2, group)
    c, qd = handle(B, kc, vc, ke, ve), q.cuda()
    kw = dict(scale=scale, max_seqlen_q=200, max_seqlen_k=900, check_status=True)
    o, lse = B.attn_kv_forward(qd, c, dev(table), dev(lens), dev(cu), **kw)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, scale, 2)
    check_attend(o, lse, ref, torch.bfloat16, 64, 900)
    for bad in (cu[:2] + [-1] + cu[3:], [x - 1 for x in cu[:-1]] + [cu[-1] + 1], cu[:-2] + [cu[-1] + 5, cu[-1]]):
        with pytest.raises(B.AttnError) as e:
            B.attn_kv_forward(qd, c, dev(table), dev(lens), dev(bad), **kw)
        assert e.value.status == B.ATTN_ERR_BAD_SEQLENS


def test_attend_long_segments_overlapping(B):
    """Padded starts that make long segments overlap: reported, nothing outside
    the declared rows touched."""
    lens, new = [80, 80, 80], [80, 80, 80]
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, lens, new, 1, 2)
    starts = dev([0, 5, 10, 90])
    out = torch.full((90, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 90), device="cuda")
    with pytest.raises(B.AttnError) as e:
        B.attn_kv_forward(q[:90].cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.1,
                          max_seqlen_q=80, max_seqlen_k=80, cu_seqlens_q_padded=starts, out=out, check_status=True)
    assert e.value.status == B.ATTN_ERR_BAD_SEQLENS


def test_attend_repeats_and_streams(B):
    """The same bits on every run, from two calls in flight on two streams, and
    from a captured graph replayed on new lengths."""
    lens, new = [3000, 1500, 7], [1, 1, 1]
    q, table, kc, vc, ke, ve, cu = attend_case(128, 128, torch.bfloat16, 16, lens, new, 2, 4)
    c, qd, td, ld, cud = handle(B, kc, vc, ke, ve), q.cuda(), dev(table), dev(lens), dev(cu)
    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=3008)
    want = B.attn_kv_forward(qd, c, td, ld, cud, **kw)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [B.attn_kv_forward(qd, c, td, ld, cud, stream=s, **kw) for _ in range(4) for s in (s1, s2)]
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    out = (torch.zeros_like(want[0]), torch.zeros_like(want[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.attn_kv_forward(qd, c, td, ld, cud, out=out, **kw)
    graph.replay()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    ld.copy_(dev([100, 900, 0]))
    graph.replay()
    ref = kv_ref.attend(q, cu, [100, 900, 0], table, kc, vc, ke, ve, 0.1, 2)
    check_attend(*out, ref, torch.bfloat16, 128, 900)


def test_offsets_past_32_bits(B):
    """A cache whose pages lie 2 GiB apart: append and attention address it with
    64 bits, keys and values past the 4 GiB mark."""
    page, heads, d, pages, gap = 16, 2, 64, 4, 1 << 31
    raw = torch.empty(pages * gap, dtype=torch.uint8, device="cuda")
    k, v = (raw.as_strided((pages, page, heads, d), (gap, heads * d, d, 1), off) for off in (0, 1 << 20))
    for x in (k, v):
        x.zero_()
    ke, ve = (torch.full((pages, heads), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    f8 = torch.float8_e4m3fn
    c = B.KvCache(k.view(f8), v.view(f8), ke, ve)
    g = torch.Generator().manual_seed(2)
    order, n = [3, 1, 2, 0], 60
    kn, vn = (torch.randn((n, heads, d), generator=g).to(torch.bfloat16) for _ in range(2))
    slots = [order[t // page] * page + t % page for t in range(n)]
    B.kv_append(kn.cuda(), vn.cuda(), dev(slots, torch.int64), c)
    kc, vc = (torch.zeros((pages, page, heads, d), dtype=torch.uint8) for _ in range(2))
    ker, ver = (torch.full((pages, heads), 127, dtype=torch.uint8) for _ in range(2))
    kv_ref.append(kc, ker, kn, slots)
    kv_ref.append(vc, ver, vn, slots)
    assert torch.equal(k.cpu(), kc) and torch.equal(v.cpu(), vc) and torch.equal(ke.cpu(), ker)
    for new in (1, 60):
        q = torch.randn((new, 4, d), generator=g).to(torch.bfloat16)
        o, lse = B.attn_kv_forward(q.cuda(), c, dev([order]), dev([n]), dev([0, new]), scale=0.125, max_seqlen_q=new,
                                   max_seqlen_k=64, check_status=True)
        check_attend(o, lse, kv_ref.attend(q, [0, new], [n], [order], kc, vc, ker, ver, 0.125, 2), torch.bfloat16, d, n,
                     weights(torch.bfloat16, new))


@pytest.mark.parametrize("heads,group,longest", [(2, 4, 1500), (1, 1, 41000)])
def test_attend_many_requests_one_long(B, heads, group, longest):
    """Over 304 jobs: few splits each, most requests with one, a long one with all
    of them (at 41,000 tokens each of its splits goes through its pages twice)."""
    g = torch.Generator().manual_seed(longest)
    batch, page, d = 320, 16, 64
    lens = torch.randint(0, 40, (batch,), generator=g).tolist()
    lens[200] = longest
    new = [1] * batch
    q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.float16, page, lens, new, heads, group)
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.125,
                               max_seqlen_q=1, max_seqlen_k=longest, check_status=True)
    check_attend(o, lse, kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.125, 2), torch.float16, d, longest)


def test_attend_nothing_to_do(B):
    """No query rows; requests without tokens; a bound of zero."""
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, [5, 9], [1, 1], 1, 2)
    c = handle(B, kc, vc, ke, ve)
    o, lse = B.attn_kv_forward(q[:0].cuda(), c, dev(table), dev([5, 9]), dev([0, 0, 0]), scale=0.1, max_seqlen_q=1,
                               max_seqlen_k=16, check_status=True)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    o, lse = B.attn_kv_forward(q.cuda(), c, dev(table), dev([0, 0]), dev(cu), scale=0.1, max_seqlen_q=1, max_seqlen_k=0,
                               check_status=True)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    B.kv_append(torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda"),
                torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda"),
                torch.empty((0,), dtype=torch.int64, device="cuda"), c)
    assert torch.equal(c.k.view(torch.uint8).cpu(), kc)


def test_attend_long_rows_the_fast_forward_does_not_take(B):
    """Segments of hundreds of tokens with a negative scale: tiles of 16 rows."""
    lens, new = [260, 150], [200, 150]
    q, table, kc, vc, ke, ve, cu = attend_case(128, 128, torch.float16, 32, lens, new, 2, 2)
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=-0.1,
                               max_seqlen_q=200, max_seqlen_k=260, check_status=True)
    check_attend(o, lse, kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, -0.1, 2), torch.float16, 128, 260)


def test_attend_window_bounds_far_out(B):
    """Window bounds near 2^31 see everything, in both paths."""
    lens, new = [90, 300], [1, 150]
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, lens, new, 1, 2)
    far = 2 ** 31 - 1
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=0.1, mask=3,
                               left=far, right=far, max_seqlen_q=150, max_seqlen_k=300, check_status=True)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, 0.1, 0)
    check_attend(o, lse, ref, torch.bfloat16, 64, 300, torch.bfloat16)


def test_what_the_binding_refuses(B):
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, [5, 9], [1, 1], 1, 2)
    c, qd, td, ld, cud = handle(B, kc, vc, ke, ve), q.cuda(), dev(table), dev([5, 9]), dev(cu)
    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=16)
    bad = [(q, c, td, ld, cud), (qd.float(), c, td, ld, cud), (qd[..., :32], c, td, ld, cud),
           (qd, c, td.long(), ld, cud), (qd, c, td.T, ld, cud), (qd, c, td, ld.long(), cud), (qd, c, td, ld, cud[:2]),
           (qd, c, td, ld, dev([[0, 1, 2]])), (qd, c, td, ld.cpu(), cud), (qd.transpose(1, 2), c, td, ld, cud)]
    for args in bad:
        with pytest.raises(ValueError):
            B.attn_kv_forward(*args, **kw)
    with pytest.raises(ValueError):
        B.attn_kv_forward(qd, c, td, ld, cud, workspace=torch.empty(10, device="cuda"), **kw)
    with pytest.raises(B.AttnError):
        B.attn_kv_forward(qd, c, td, ld, cud, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw)
    k = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    sl = dev([0, 1], torch.int64)
    for args in ((k, k, sl.int(), c), (k, k[:1], sl, c), (k.half(), k, sl, c), (k.float(), k.float(), sl, c),
                 (k, k.cpu(), sl, c), (k, k, sl[:1], c)):
        with pytest.raises(ValueError):
            B.kv_append(*args)
    one = dev([1, 1])
    plan = dict(page_size=16, max_tokens=4)
    for args in ((one, ld.long(), td, dev([0, 1]), dev([0])), (one, ld[:1], td, dev([0, 1]), dev([0])),
                 (one, ld, td.T, dev([0, 1]), dev([0])), (one, ld, td, dev([0, 1]), dev([0, 0])),
                 (one, ld, td, dev([0, 1]).cpu(), dev([0]))):
        with pytest.raises(ValueError):
            B.kv_plan(*args, **plan)
    f = B.rope_frequencies(64)
    pos = dev([1, 2])
    for args in ((qd, None, pos.long(), f), (qd, None, pos[:1], f), (qd, None, pos.cpu(), f), (qd, None, pos, f.float()),
                 (qd, None, pos, f.cuda()), (qd, qd[..., :32], pos, f), (qd, qd.half(), pos, f),
                 (qd.transpose(1, 2), None, pos, f), (qd[0], None, pos, f)):
        with pytest.raises((ValueError, B.AttnError)):
            B.rope(*args)


def test_expanded_tensors_are_refused(B):
    """Strides of zero in a tensor with more than one entry: the library would
    take three of them for contiguous and read past the tensor."""
    def e(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape[-1], dtype=dtype, device="cuda").expand(shape)

    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, [5, 9], [1, 1], 1, 2)
    c, qd, td, ld, cud = handle(B, kc, vc, ke, ve), q.cuda(), dev(table), dev([5, 9]), dev(cu)
    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=16)
    flat = torch.zeros_like(qd)
    lse = torch.zeros((qd.shape[1], qd.shape[0]), device="cuda")
    for x in (e(*qd.shape), qd[:1].expand(qd.shape), qd[:, :1].expand(qd.shape)):
        with pytest.raises(ValueError, match="expanded"):
            B.attn_kv_forward(x, c, td, ld, cud, **kw)
        with pytest.raises(ValueError, match="expanded"):
            B.attn_kv_forward(qd, c, td, ld, cud, out=(x, lse), **kw)
        with pytest.raises(ValueError, match="expanded"):
            B.rope(x, None, dev([1, 2]), B.rope_frequencies(64))
        with pytest.raises(ValueError, match="expanded"):
            B.rope(flat, x, dev([1, 2]), B.rope_frequencies(64))
        with pytest.raises(ValueError, match="expanded"):
            B.rope(flat, None, dev([1, 2]), B.rope_frequencies(64), out=(x, None))
    k, sl = torch.zeros((2, c.nhead_kv, 64), dtype=torch.bfloat16, device="cuda"), dev([0, 1], torch.int64)
    for args in ((e(2, c.nhead_kv, 64), k), (k, e(2, c.nhead_kv, 64))):
        with pytest.raises(ValueError, match="expanded"):
            B.kv_append(*args, sl, c)
    page, byte = e(4, 16, 2, 64, dtype=torch.uint8), torch.zeros((4, 16, 2, 64), dtype=torch.uint8, device="cuda")
    s = torch.full((4, 2), 127, dtype=torch.uint8, device="cuda")
    for args in ((page, byte), (byte, page)):
        with pytest.raises(ValueError, match="expanded"):
            B.KvCache(*args, s, s.clone())
    # one entry may carry any stride
    assert torch.equal(B.rope(flat[:1, :1].expand(1, 1, 64), None, dev([1]), B.rope_frequencies(64))[0], flat[:1, :1])


def test_a_cache_handle_keeps_its_tensors(B):
    c = B.KvCache.empty(4, 16, 2, 64, 64)
    for name in ("k", "v", "k_exp", "v_exp", "packed", "page_size"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))


# ------------------------------------------------------- the step they make up

@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(B, graph):
    """plan -> rope -> append -> attend over several steps: prompts, decoding,
    a request that leaves and one that takes its pages; every step's cache
    bytes, bookkeeping and attention against the oracle's.  Captured, the same
    graph replays each step on new inputs."""
    page, hkv, group, d, batch, pool, cols, cap = 16, 2, 4, 64, 3, 14, 8, 64
    dtype, scale = torch.bfloat16, 64 ** -0.5
    g = torch.Generator().manual_seed(11)
    steps = [[20, 0, 33], [1, 17, 1], [1, 1, 1], [-1, 2, 1], [40, 1, 0], [1, 1, -1], [0, 1, 0]]
    f, axis = B.rope_frequencies(d), (torch.arange(d // 2) % 2).to(torch.uint8)
    # the oracle's state and the device's
    lens, table, free, count = [0] * batch, [[-1] * cols for _ in range(batch)], list(range(pool)), pool
    kc, vc = (torch.zeros((pool, page, hkv, d), dtype=torch.uint8) for _ in range(2))
    ke, ve = (torch.full((pool, hkv), 127, dtype=torch.uint8) for _ in range(2))
    c = handle(B, kc, vc, ke, ve)
    td, fd, ld, cd, nd = dev(table), dev(free), dev(lens), dev([count]), dev([0] * batch)
    qd = torch.zeros((cap, hkv * group, d), dtype=dtype, device="cuda")
    kd, vd = (torch.zeros((cap, hkv, d), dtype=dtype, device="cuda") for _ in range(2))
    hd = torch.zeros(cap, dtype=I32, device="cuda")          # a second axis, from the program
    out = B.KvPlan(torch.empty(batch + 1, dtype=I32, device="cuda"), ld, torch.empty(cap, dtype=I32, device="cuda"),
                   torch.empty(cap, dtype=torch.int64, device="cuda"), cd, dev([0]))
    both = torch.empty((2, cap), dtype=I32, device="cuda")

    def step():
        p = B.kv_plan(nd, ld, td, fd, cd, page_size=page, max_tokens=cap, out=out)
        both[0].copy_(p.positions)
        both[1].copy_(hd)
        rq, rk = B.rope(qd, kd, both, f, pair_axis=axis)
        B.kv_append(rk, vd, p.slots, c)
        o, lse = B.attn_kv_forward(rq, c, td, p.seqlens, p.cu_seqlens, scale=scale, max_seqlen_q=48,
                                   max_seqlen_k=cols * page)
        return rq, rk, o, lse

    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            held = step()
    for new in steps:
        n = sum(max(x, 0) for x in new)
        q = torch.randn((cap, hkv * group, d), generator=g).to(dtype)
        k, v = (torch.randn((cap, hkv, d), generator=g).to(dtype) for _ in range(2))
        h2 = torch.randint(0, 9, (cap,), generator=g, dtype=I32)
        for dst, src in ((qd, q), (kd, k), (vd, v), (hd, h2), (nd, torch.tensor(new, dtype=I32))):
            dst.copy_(src)
        if graph:
            gr.replay()
            rq, rk, o, lse = held
        else:
            rq, rk, o, lse = step()
        torch.cuda.synchronize()
        out.check()
        cu, lens, pos, slots, count = kv_ref.plan(new, lens, table, free, count, page, cap)
        assert ld.tolist() == lens and cd.tolist() == [count] and td.tolist() == table and out.slots.tolist() == slots
        pp = torch.stack([torch.tensor(pos, dtype=I32), h2])
        for x, got in ((q, rq), (k, rk)):
            ref = kv_ref.rope(x, pp, f, axis)
            assert float((got.cpu().to(torch.float64) - ref).abs().max()) <= 2.0 ** -8 * 6   # half a step below 6
        # from the device's own rounded keys and queries on, so that both sides store the same bytes
        kv_ref.append(kc, ke, rk.cpu(), slots)
        kv_ref.append(vc, ve, v, slots)
        for got, ref in ((c.k, kc), (c.v, vc), (c.k_exp, ke), (c.v_exp, ve)):
            assert torch.equal(got.view(torch.uint8).cpu(), ref)
        if n:
            ref = kv_ref.attend(rq.cpu()[:n], cu, lens, table, kc, vc, ke, ve, scale, 2)
            check_attend(o[:n], lse[:, :n], ref, dtype, d, max(lens), weights(dtype, max(new)))
