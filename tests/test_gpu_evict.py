"""Accumulated attention weights and eviction on the GPU against the fp64 oracle,
alone and in the serving loop that they make up with the cache's other operators."""
import math

import pytest
import torch

from oracle import evict_ref, kv_ref
from tests.kv_cases import block_table, check_attend, random_cache
from tests.test_gpu_kv import dev, handle
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

I32, F64 = torch.int32, torch.float64


def weights_of(B, weight, position):
    return B.KvWeights(weight.cuda(), position.cuda(), torch.zeros(1, dtype=I32, device="cuda"))


def random_weights(pages, heads, page, g):
    return (2 * torch.randn((pages, heads, page), generator=g)).exp(), torch.randint(0, 500, (pages, heads, page), generator=g).to(I32)


# --------------------------------------------------------------------- weigh

def weigh_case(B, dtype, lens, new, page, hkv, group, d, dv=None, mask=2, left=-1, right=-1, decay=1.0, seed=0, scale=None,
               padded=False, offsets=True, tight=True, fresh=None):
    """Runs one call and compares; the kernel's error per weight is at most the sum of
    p (score error + exponent's argument and ex2, 2^-22 (|s| + |LSE| + 1)) over its rows,
    plus one rounding per addition (the oracle returns that bound)."""
    g = torch.Generator().manual_seed(seed + sum(lens) + d)
    dv = d if dv is None else dv
    table, pool = block_table(lens, page, g)
    kc, ke = random_cache(pool, page, hkv, d, g)
    vc, ve = random_cache(pool, page, hkv, dv, g)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    starts, total = list(cu[:-1]), cu[-1]
    if padded:
        starts, total = [], 0
        for n in new:
            starts.append(total + 2)
            total += n + 3
    hq = hkv * group
    q = torch.randn((total + 1, hq, d), generator=g).to(dtype)
    scale = d ** -0.5 if scale is None else scale
    # the packed rows' LSE, from the oracle; other rows hold anything
    rows = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, new)]) if sum(new) else torch.zeros(0, dtype=torch.long)
    _, lse_packed, _, _ = kv_ref.attend(q[rows], cu, lens, table, kc, vc, ke, ve, scale, mask, left, right)
    lse = torch.full((hq, total + 1), math.nan)
    lse[:, rows] = lse_packed.float()
    weight, position = random_weights(pool, hkv, page, g)
    off = [7 * b + 1 for b in range(len(lens))] if offsets else [0] * len(lens)
    want, where, slack = evict_ref.weigh(q[rows], lse[:, rows], cu, lens, table, kc, ke, weight, position, off, scale, mask, left,
                                         right, decay, fresh)
    c = handle(B, kc, vc, ke, ve)
    w = weights_of(B, weight, position)
    kw = dict(scale=scale, mask=mask, left=left, right=right, decay=decay, max_seqlen_q=max(new) if tight else 1000,
              max_seqlen_k=max(lens) if tight else len(table[0]) * page,
              position_offsets=dev(off) if offsets else None, new_lens=dev(fresh) if fresh else None,
              cu_seqlens_q_padded=dev(starts + [total]) if padded else None)
    B.kv_weigh(q.cuda(), lse.cuda(), c, w, dev(table), dev(lens), dev(cu), **kw)
    w.check()
    got = w.weight.cpu().to(F64)
    assert torch.equal(w.position.cpu(), where)
    bad = (got - want).abs() > slack
    assert not bool(bad.any()), f"{int(bad.sum())} weights off, by up to {float((got - want).abs().max())}"
    again = weights_of(B, weight, position)
    B.kv_weigh(q.cuda(), lse.cuda(), c, again, dev(table), dev(lens), dev(cu), **kw)
    assert torch.equal(again.weight, w.weight)
    return w


WEIGHS = [
    # lens, new, page, kv heads, group, d, d_v
    ([1], [1], 16, 1, 1, 64, 64), ([1, 0, 17], [1, 0, 1], 16, 2, 4, 128, 128), ([100, 33, 64, 5], [1, 1, 0, 5], 32, 3, 2, 64, 64),
    ([257, 16], [3, 16], 16, 2, 3, 192, 128), ([300], [40], 128, 1, 8, 256, 256), ([520, 129], [70, 129], 16, 2, 2, 128, 128),
    ([1000], [1], 256, 2, 1, 128, 128), ([2100, 40], [1, 1], 16, 2, 4, 128, 128), ([150], [150], 64, 1, 16, 64, 64),
]


@pytest.mark.parametrize("lens,new,page,hkv,group,d,dv", WEIGHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weigh(B, lens, new, page, hkv, group, d, dv, dtype):
    weigh_case(B, dtype, lens, new, page, hkv, group, d, dv)


@pytest.mark.parametrize("mask,left,right", [(0, -1, -1), (1, -1, -1), (3, 20, 0), (3, 0, -1), (3, 5, 3), (3, -1, -1)])
@pytest.mark.parametrize("decay", [1.0, 0.75, 0.0])
def test_weigh_masks_and_decay(B, mask, left, right, decay):
    weigh_case(B, torch.bfloat16, [130, 70, 33], [5, 1, 33], 16, 2, 2, 64, 64, mask, left, right, decay)


@pytest.mark.parametrize("mask,left", [(0, -1), (1, -1), (2, -1), (3, 20)])
@pytest.mark.parametrize("new", [[1, 4, 0, 2], [70, 4, 0, 90]])
@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_weigh_new_lens(B, mask, left, new, decay):
    """Fewer or more tokens are new than query: whole prompts that their last queries
    weigh, tokens weighed before, none.  Both kernels."""
    weigh_case(B, torch.bfloat16, [150, 70, 33, 300], new, 16, 2, 2, 64, 64, mask, left, 0 if mask == 3 else -1, decay,
               fresh=[150, 0, 33, 217])


def test_weigh_reports_new_lens(B):
    g, table, pool, kc, ke, vc, ve = small(B)
    q, lse = torch.randn((2, 4, 64), generator=g).bfloat16().cuda(), torch.full((4, 2), 3.0, device="cuda")
    weight, position = random_weights(pool, 2, 16, g)
    for bad in ([-1, 1], [51, 1]):
        w = weights_of(B, weight, position)
        B.kv_weigh(q, lse, handle(B, kc, vc, ke, ve), w, dev(table), dev([50, 20]), dev([0, 1, 2]), scale=0.1, new_lens=dev(bad),
                   max_seqlen_q=1, max_seqlen_k=64)
        with pytest.raises(B.AttnError) as e:
            w.check()
        assert e.value.status == B.ATTN_ERR_BAD_SEQLENS
        for j in range(50):
            assert torch.equal(w.weight[table[0][j // 16], :, j % 16].cpu(), weight[table[0][j // 16], :, j % 16])
        assert not torch.equal(w.weight[table[1][0]].cpu(), weight[table[1][0]])


LONG_WEIGHS = [
    # lens, new, page, kv heads, group, d, d_v, mask, left, right
    ([1500, 130], [700, 129], 16, 1, 4, 128, 128, 2, -1, -1), ([260], [260], 64, 2, 3, 64, 64, 2, -1, -1),
    ([300, 1000, 77], [200, 1, 30], 32, 2, 5, 192, 128, 2, -1, -1), ([129, 600], [128, 140], 256, 1, 2, 256, 256, 2, -1, -1),
    ([700], [300], 16, 2, 1, 128, 128, 3, 100, 0), ([700, 300], [90, 300], 16, 1, 2, 64, 64, 3, 33, 17),
    ([400], [200], 16, 1, 128, 64, 64, 2, -1, -1), ([140], [30], 16, 1, 70, 192, 128, 2, -1, -1), ([130, 500], [90, 260], 128, 2, 2, 128, 128, 0, -1, -1),
    ([90, 40], [200, 100], 16, 1, 2, 128, 128, 2, -1, -1), ([330], [140], 16, 1, 2, 128, 128, 1, -1, -1),
]


@pytest.mark.parametrize("lens,new,page,hkv,group,d,dv,mask,left,right", LONG_WEIGHS)
@pytest.mark.parametrize("dtype,decay", [(torch.bfloat16, 1.0), (torch.float16, 0.5)])
def test_weigh_long_segments(B, lens, new, page, hkv, group, d, dv, mask, left, right, dtype, decay):
    weigh_case(B, dtype, lens, new, page, hkv, group, d, dv, mask, left, right, decay, padded=decay != 1.0)


def test_weigh_long_segment_rows_without_a_finite_lse(B):
    """A query row of NaN in a long segment, and padding rows of NaN behind the last one."""
    g, table, pool, kc, ke, vc, ve = small(B, lens=(200, 20), d=128)
    q = torch.randn((150, 4, 128), generator=g).bfloat16()
    lse = torch.full((4, 150), 3.0)
    q[7, 1], lse[1, 7] = math.nan, math.nan
    q[141:], lse[:, 141:] = math.nan, math.nan
    lse[2, 30] = -math.inf
    weight, position = random_weights(pool, 2, 16, g)
    w = weights_of(B, weight, position)
    B.kv_weigh(q.cuda(), lse.cuda(), handle(B, kc, vc, ke, ve), w, dev(table), dev([200, 20]), dev([0, 140, 141]), scale=0.08,
               max_seqlen_q=140, max_seqlen_k=208)
    w.check()
    q[7, 1] = 0
    want, where, slack = evict_ref.weigh(q, lse, [0, 140, 141], [200, 20], table, kc, ke, weight, position, [0, 0], 0.08)
    assert bool(((w.weight.cpu().double() - want).abs() <= slack).all()) and torch.equal(w.position.cpu(), where)


def test_weigh_long_segment_reports_pages(B):
    g, table, pool, kc, ke, vc, ve = small(B, lens=(200, 20), d=64)
    c = handle(B, kc, vc, ke, ve)
    q, lse = torch.randn((120, 4, 64), generator=g).bfloat16().cuda(), torch.full((4, 120), 3.0, device="cuda")
    weight, position = random_weights(pool, 2, 16, g)
    good, w = weights_of(B, weight, position), weights_of(B, weight, position)
    kw = dict(scale=0.08, max_seqlen_q=120, max_seqlen_k=208)
    B.kv_weigh(q, lse, c, good, dev(table), dev([200, 20]), dev([0, 119, 120]), **kw)
    good.check()
    broken = [list(r) for r in table]
    broken[0][5] = pool
    B.kv_weigh(q, lse, c, w, dev(broken), dev([200, 20]), dev([0, 119, 120]), **kw)
    with pytest.raises(B.AttnError) as e:
        w.check()
    assert e.value.status == B.ATTN_ERR_BAD_PAGE
    same = [p for p in range(pool) if p != table[0][5]]
    assert torch.equal(w.weight[same], good.weight[same])
    assert torch.equal(w.weight[table[0][5]].cpu(), weight[table[0][5]])


def test_weigh_more_queries_than_keys(B):
    """Rows that see nothing have LSE = -inf and add nothing."""
    weigh_case(B, torch.bfloat16, [10, 200], [30, 210], 16, 2, 2, 64)


def test_weigh_padded_segments_and_loose_bounds(B):
    weigh_case(B, torch.float16, [100, 0, 65], [3, 0, 1], 16, 2, 4, 128, padded=True, tight=False)
    weigh_case(B, torch.float16, [100, 12, 165], [50, 1, 165], 16, 2, 2, 128, padded=True, tight=False, offsets=False)


def test_weigh_negative_scale(B):
    weigh_case(B, torch.bfloat16, [90], [2], 16, 1, 2, 64, scale=-0.1)
    weigh_case(B, torch.bfloat16, [190], [100], 16, 1, 2, 64, scale=-0.1)


def small(B, seed=1, lens=(50, 20), page=16, hkv=2, d=64):
    g = torch.Generator().manual_seed(seed)
    table, pool = block_table(list(lens), page, g)
    kc, ke = random_cache(pool, page, hkv, d, g)
    vc, ve = random_cache(pool, page, hkv, d, g)
    return g, table, pool, kc, ke, vc, ve


def test_weigh_rows_without_a_finite_lse_and_nan_keys(B):
    g, table, pool, kc, ke, vc, ve = small(B)
    kc[table[0][1], 3, 0] = 127                      # NaN in one key of one head
    kc[table[0][3], 2:, :] = 127                     # rows past the end: no key of the request
    q = torch.randn((4, 4, 64), generator=g).bfloat16()
    lse = torch.full((4, 4), 3.0)
    lse[0, 1], lse[1, 0], lse[2, 2] = math.nan, -math.inf, math.inf
    weight, position = random_weights(pool, 2, 16, g)
    w = weights_of(B, weight, position)
    kw = dict(scale=0.125, max_seqlen_q=2, max_seqlen_k=64)
    B.kv_weigh(q.cuda(), lse.cuda(), handle(B, kc, vc, ke, ve), w, dev(table), dev([50, 20]), dev([0, 2, 4]), **kw)
    w.check()
    got = w.weight.cpu()
    assert math.isnan(float(got[table[0][1], 0, 3]))
    got[table[0][1], 0, 3] = 0.0
    assert bool(torch.isfinite(got).all())
    kc2 = kc.clone()
    kc2[table[0][1], 3, 0] = 0
    kc2[table[0][3], 2:, :] = 0
    want, where, slack = evict_ref.weigh(q, lse, [0, 2, 4], [50, 20], table, kc2, ke, weight, position, [0, 0], 0.125)
    want[table[0][1], 0, 3] = 0.0
    assert bool(((got.double() - want).abs() <= slack + 1e-30).all()) and torch.equal(w.position.cpu(), where)


@pytest.mark.parametrize("lq", [1, 30, 140])
@pytest.mark.parametrize("layout", ["heads outside rows", "a part of wider rows"])
def test_weigh_strided_queries_and_streams(B, lq, layout):
    """The bits of the contiguous call, on a stream that is given or current."""
    g, table, pool, kc, ke, vc, ve = small(B, lens=(200, 20), d=128)
    q = torch.randn((lq + 1, 4, 128), generator=g).bfloat16().cuda()
    lse = torch.full((4, lq + 1), 5.0, device="cuda")
    c = handle(B, kc, vc, ke, ve)
    if layout == "heads outside rows":
        strided = q.transpose(0, 1).contiguous().transpose(0, 1)
    else:
        strided = torch.full((lq + 1, 8, 128), math.nan, device="cuda").bfloat16()[:, 2:6]
        strided.copy_(q)
    assert not strided.is_contiguous() or lq == 0
    td, ld, cu = dev(table), dev([200, 20]), dev([0, lq, lq + 1])
    weight, position = random_weights(pool, 2, 16, g)
    kw = dict(scale=0.08, max_seqlen_q=lq, max_seqlen_k=208)
    a, b, d = weights_of(B, weight, position), weights_of(B, weight, position), weights_of(B, weight, position)
    B.kv_weigh(q, lse, c, a, td, ld, cu, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.kv_weigh(strided, lse, c, b, td, ld, cu, stream=side, **kw)
    with torch.cuda.stream(side):
        B.kv_weigh(strided, lse, c, d, td, ld, cu, **kw)
    side.synchronize()
    for w in (a, b, d):
        w.check()
        assert torch.equal(w.weight, a.weight) and torch.equal(w.position, a.position)
    assert not torch.equal(a.weight.cpu(), weight)


@pytest.mark.parametrize("lq,window", [(1, 0), (3, 0), (30, 0), (140, 0), (30, 20), (140, 60)])
def test_weigh_nan_key_after_a_forward(B, lq, window):
    """A NaN in a key makes the LSE of every row that sees it NaN, in its kv head: those
    rows add nothing, to that key neither, whichever kernel the segment's length takes."""
    g, table, pool, kc, ke, vc, ve = small(B, lens=(200, 20))
    kc[table[0][10], 3, 0] = 127                     # key 163
    q = torch.randn((lq + 1, 4, 64), generator=g).bfloat16()
    c, cu, kw = handle(B, kc, vc, ke, ve), [0, lq, lq + 1], dict(scale=0.125, max_seqlen_q=lq, max_seqlen_k=208)
    kw.update(mask=3, left=window, right=0) if window else kw.update(mask=2)
    lse = B.attn_kv_forward(q.cuda(), c, dev(table), dev([200, 20]), dev(cu), **kw)[1]
    weight, position = random_weights(pool, 2, 16, g)
    w = weights_of(B, weight, position)
    B.kv_weigh(q.cuda(), lse, c, w, dev(table), dev([200, 20]), dev(cu), **kw)
    w.check()
    assert bool(torch.isnan(lse[:2, :lq]).any()) and bool(torch.isfinite(lse[2:]).all())
    kc[table[0][10], 3, 0] = 0
    want, where, slack = evict_ref.weigh(q, lse.cpu(), cu, [200, 20], table, kc, ke, weight, position, [0, 0], 0.125,
                                         mask=kw["mask"], left=window or -1, right=0 if window else -1)
    assert bool(((w.weight.cpu().double() - want).abs() <= slack + 1e-30).all()) and torch.equal(w.position.cpu(), where)


def test_weigh_decay_zero_does_not_read(B):
    g, table, pool, kc, ke, vc, ve = small(B)
    q = torch.randn((2, 4, 64), generator=g).bfloat16().cuda()
    w = weights_of(B, torch.full((pool, 2, 16), math.nan), torch.zeros((pool, 2, 16), dtype=I32))
    B.kv_weigh(q, torch.full((4, 2), 3.0, device="cuda"), handle(B, kc, vc, ke, ve), w, dev(table), dev([50, 20]), dev([0, 1, 2]),
               scale=0.125, decay=0.0, max_seqlen_q=1, max_seqlen_k=64)
    got = w.weight.cpu()
    for b, n in enumerate((50, 20)):
        for j in range(n):
            assert bool(torch.isfinite(got[table[b][j // 16], :, j % 16]).all())
    assert int(torch.isnan(got).sum()) == (pool * 16 - 70) * 2


def test_weigh_reports_lengths_and_pages(B):
    g, table, pool, kc, ke, vc, ve = small(B, lens=(50, 20, 40))
    c = handle(B, kc, vc, ke, ve)
    q = torch.randn((3, 4, 64), generator=g).bfloat16().cuda()
    lse = torch.full((4, 3), 3.0, device="cuda")
    weight, position = random_weights(pool, 2, 16, g)
    run = lambda w, table, lens, cu, **kw: B.kv_weigh(q, lse, c, w, dev(table), dev(lens), dev(cu),   # noqa: E731
                                                      **{**dict(scale=0.125, max_seqlen_q=1, max_seqlen_k=64), **kw})
    good = weights_of(B, weight, position)
    run(good, table, [50, 20, 40], [0, 1, 2, 3])
    good.check()
    rows = [(b, j) for b, n in enumerate((50, 20, 40)) for j in range(n)]
    for lens, cu, lost in (([50, -1, 40], [0, 1, 2, 3], 1), ([50, 65, 40], [0, 1, 2, 3], 1), ([50, 20, 40], [0, 1, 3, 4], 1),
                           ([50, 20, 40], [0, 1, 0, 1], 1)):
        w = weights_of(B, weight, position)
        run(w, table, lens, cu)
        with pytest.raises(B.AttnError) as e:
            w.check()
        assert e.value.status == B.ATTN_ERR_BAD_SEQLENS
        for b, j in rows:
            at = (table[b][j // 16], slice(None), j % 16)
            if b == lost:
                assert torch.equal(w.weight[at].cpu(), weight[at])
            elif cu == [0, 1, 2, 3]:
                assert torch.equal(w.weight[at], good.weight[at])
    for bad in (-1, pool, 2 ** 30):
        broken = [list(r) for r in table]
        broken[0][1] = bad
        w = weights_of(B, weight, position)
        run(w, broken, [50, 20, 40], [0, 1, 2, 3])
        with pytest.raises(B.AttnError) as e:
            w.check()
        assert e.value.status == B.ATTN_ERR_BAD_PAGE
        for b, j in rows:
            at = (table[b][j // 16], slice(None), j % 16)
            if (b, j // 16) == (0, 1):
                assert torch.equal(w.weight[at].cpu(), weight[at])
            else:
                assert torch.equal(w.weight[at], good.weight[at])


def test_refused_tensors(B):
    g, table, pool, kc, ke, vc, ve = small(B)
    c = handle(B, kc, vc, ke, ve)
    w = B.KvWeights.empty(c)
    q, lse = torch.zeros((2, 4, 64), device="cuda").bfloat16(), torch.zeros((4, 2), device="cuda")
    td, ld, cu = dev(table), dev([50, 20]), dev([0, 1, 2])
    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=64)
    for args in ((q.float(), lse, c, w, td, ld, cu), (q, lse.double(), c, w, td, ld, cu), (q, lse[:, :1], c, w, td, ld, cu),
                 (q, lse, c, w._replace(weight=w.weight[:, :1]), td, ld, cu), (q, lse, c, w._replace(position=w.weight), td, ld, cu),
                 (q, lse, c, w, td[:1], ld, cu), (q, lse, c, w, td, ld, cu[:2]), (q[:, :, :32], lse, c, w, td, ld, cu),
                 (q, lse, c, tuple(w)[:2], td, ld, cu), (q, lse, c, w, td.long(), ld, cu), (q.cpu(), lse, c, w, td, ld, cu)):
        with pytest.raises(ValueError):
            B.kv_weigh(*args, **kw)
    with pytest.raises(B.AttnError):
        B.kv_weigh(q, lse, c, w, td, ld, cu, **{**kw, "decay": -1.0})
    keep, off, free, count = dev([10, 10]), dev([0, 0]), dev([0] * pool), dev([0])
    for args in ((c, w, keep[:1], ld, off, td, free, count), (c, w, keep, ld, off, td, free[:-1], count),
                 (c, w, keep, ld, off.float(), td, free, count), (c, w._replace(weight=w.weight.half()), keep, ld, off, td, free, count)):
        with pytest.raises(ValueError):
            B.kv_evict(*args, max_seqlen_k=64)
    with pytest.raises(B.AttnError) as e:
        B.kv_evict(c, w, keep, ld, off, td, free, count, max_seqlen_k=64, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B.ATTN_ERR_WORKSPACE_TOO_SMALL


# --------------------------------------------------------------------- evict

def evict_case(B, lens, keep, page, hkv, d, dv, sink=0, recent=0, slack=0, seed=0, spread=3, change=None, in_place=False,
               bound=None):
    g = torch.Generator().manual_seed(seed + sum(lens))
    table, pool = block_table(lens, page, g, extra_pages=3)
    kc, ke = random_cache(pool, page, hkv, d, g, spread)
    vc, ve = random_cache(pool, page, hkv, dv, g, spread)
    weight, position = random_weights(pool, hkv, page, g)
    offsets = torch.randint(0, 50, (len(lens),), generator=g).tolist()
    if change:
        change(weight, position, table)
    used = {p for r in table for p in r if p >= 0}
    free = [p for p in range(pool) if p not in used]
    count = len(free)
    free += [-5] * (pool - count)
    c, w = handle(B, kc, vc, ke, ve), weights_of(B, weight, position)
    kd, ld, od, td, fd, cd = dev(keep), dev(lens), dev(offsets), dev(table), dev(free), dev([count])
    out = B.KvEviction(ld, od, cd, dev([9])) if in_place else None
    e = B.kv_evict(c, w, kd, ld, od, td, fd, cd, sink=sink, recent=recent, slack=slack, max_seqlen_k=bound or max(max(lens), 1), out=out)
    e.check()
    if not in_place:
        assert ld.tolist() == lens and od.tolist() == offsets and cd.tolist() == [count]
    cache, exps = {"k": kc, "v": vc}, {"k": ke, "v": ve}
    after, forgotten, left = evict_ref.evict(keep, lens, offsets, table, free, count, cache, exps, weight, position, sink, recent,
                                             slack)
    assert e.seqlens.tolist() == after and e.position_offsets.tolist() == forgotten and e.free_count.tolist() == [left]
    assert fd.tolist() == free and td.tolist() == table
    for got, ref in ((c.k, kc), (c.v, vc), (c.k_exp, ke), (c.v_exp, ve)):
        assert torch.equal(got.view(torch.uint8).cpu(), ref)
    assert torch.equal(w.weight.cpu().view(I32), weight.view(I32)) and torch.equal(w.position.cpu(), position)


EVICTS = [
    # lens, keep, page, kv heads, d, d_v
    ([1], [0], 16, 1, 64, 64), ([40], [39], 16, 2, 64, 64), ([17, 16, 33], [16, 16, 1], 16, 2, 128, 128),
    ([100, 0, 64, 5], [37, 5, -1, 4], 32, 2, 64, 64), ([300, 290], [128, 64], 64, 1, 192, 128), ([500], [77], 256, 2, 64, 64),
    ([130, 70], [0, 66], 16, 2, 256, 256), ([700], [699], 16, 1, 64, 64),
]


@pytest.mark.parametrize("lens,keep,page,hkv,d,dv", EVICTS)
@pytest.mark.parametrize("sink,recent", [(0, 0), (20, 450), (500, 0)])
def test_evict(B, lens, keep, page, hkv, d, dv, sink, recent):
    evict_case(B, lens, keep, page, hkv, d, dv, sink, recent)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("spread", [1, 14])
def test_evict_scales_and_outputs(B, in_place, spread):
    """One scale everywhere (bytes move as they are), and scales that differ by up to 2^13."""
    evict_case(B, [200, 90], [100, 50], 16, 2, 128, 128, spread=spread, in_place=in_place, bound=1000)


def test_evict_slack(B):
    evict_case(B, [70, 71, 75], [60, 60, 60], 16, 1, 64, 64, slack=10)


@pytest.mark.parametrize("steps", [1, 3, 50])
def test_evict_few_distinct_weights(B, steps):
    """Ties at every digit: all of a key's rows stay, some, or the first alone."""
    def few(weight, position, table):
        weight.copy_((torch.randint(0, steps, weight.shape, generator=torch.Generator().manual_seed(steps)) + 1) * 2.0 ** -11 + 1)
        position.fill_(1 << 20)
        position[::2] = -5
    for keep in (1, 40, 99, 149):
        evict_case(B, [150, 60], [keep, 30], 16, 2, 64, 64, change=few)
        evict_case(B, [150, 60], [keep, 30], 16, 2, 64, 64, sink=1, change=few)


def test_evict_equal_weights_and_odd_ones(B):
    def equal(weight, position, table):
        weight.fill_(1.0)
        position.fill_(100)
    evict_case(B, [150, 33], [70, 10], 16, 2, 64, 64, change=equal)

    def odd(weight, position, table):
        weight[:, :, ::3] = math.nan
        weight[:, :, 1::5] = -0.0
        weight[:, :, 2::7] = math.inf
        weight[:, :, 4::7] = -math.inf
        weight[:, :, 6::7] = -1.0
        weight[:, :, 7::8] = 1e-42
    evict_case(B, [150, 33], [70, 10], 16, 2, 64, 64, sink=30, change=odd)
    evict_case(B, [150, 33], [140, 30], 16, 2, 64, 64, change=odd)


@pytest.mark.parametrize("n,keep", [(8193, 4000), (20000, 19990), (50000, 1000)])
def test_evict_by_clusters(B, n, keep):
    evict_case(B, [n, 300], [keep, 100], 64, 1, 64, 64, sink=10, recent=600, bound=n)


def big_evict(B, n, keep, page, change):
    """One head; the choice, the moves and the stack against torch's stable sort."""
    g = torch.Generator().manual_seed(n)
    pages = (n + page - 1) // page
    order = torch.randperm(pages, generator=g)
    kc = torch.randint(0, 120, (pages, page, 1, 64), generator=g, dtype=torch.uint8)
    ke = torch.full((pages, 1), 120, dtype=torch.uint8)
    weight, position = random_weights(pages, 1, page, g)
    change(weight)
    c, w = handle(B, kc, kc.clone(), ke, ke.clone()), weights_of(B, weight, position)
    free, count = dev([0] * pages), dev([0])
    e = B.kv_evict(c, w, dev([keep]), dev([n]), dev([1000]), order.to(I32)[None].cuda(), free, count, max_seqlen_k=pages * page)
    e.check()
    flat = weight[order, 0].flatten()[:n]
    kept = torch.zeros(n, dtype=torch.bool)
    kept[flat.sort(descending=True, stable=True).indices[:keep]] = True
    to, frm = torch.nonzero(~kept[:keep])[:, 0], torch.nonzero(kept[keep:])[:, 0] + keep
    rows = kc[order, :, 0].flatten(0, 1)
    rows[to] = rows[frm]
    flat[to] = flat[frm]
    assert torch.equal(c.k.view(torch.uint8).cpu()[order, :, 0].flatten(0, 1), rows)
    assert torch.equal(c.v.view(torch.uint8).cpu()[order, :, 0].flatten(0, 1), rows)
    assert torch.equal(w.weight.cpu()[order, 0].flatten()[:n], flat)
    need = (keep + page - 1) // page
    assert e.free_count.tolist() == [pages - need] and torch.equal(free.cpu()[: pages - need], order[need:].to(I32))


def test_evict_more_rows_than_shared_memory_holds(B):
    big_evict(B, 330001, 100003, 16, lambda w: None)
    big_evict(B, 400000, 399000, 256, lambda w: w.mul_(4).round_())       # many equal weights


@pytest.mark.parametrize("what,status", [
    ("len below zero", -7), ("len past the bound", -7), ("keep below -1", -7), ("free_count negative", -7),
    ("free_count past the pool", -7), ("stack too full", -7), ("bad page", -8), ("page past the pool", -8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_refused_call_changes_nothing(B, what, status, in_place):
    g = torch.Generator().manual_seed(3)
    lens, keep, count = [60, 50, 20], [20, 10, -1], 3
    table, pool = block_table(lens, 16, g, extra_pages=3)
    if what == "len below zero":
        lens[2] = -1
    elif what == "len past the bound":
        lens[0] = 65
    elif what == "keep below -1":
        keep[2] = -2
    elif what == "free_count negative":
        count = -1
    elif what == "free_count past the pool":
        count = pool + 1
    elif what == "stack too full":
        count = pool - 3
    elif what == "bad page":
        table[1][3] = -1
    elif what == "page past the pool":
        table[0][0] = pool
    kc, ke = random_cache(pool, 16, 2, 64, g)
    vc, ve = random_cache(pool, 16, 2, 64, g)
    weight, position = random_weights(pool, 2, 16, g)
    c, w = handle(B, kc, vc, ke, ve), weights_of(B, weight, position)
    free = list(range(100, 100 + pool))
    kd, ld, od, td, fd, cd = dev(keep), dev(lens), dev([4, 5, 6]), dev(table), dev(free), dev([count])
    out = B.KvEviction(ld, od, cd, dev([9])) if in_place else None
    e = B.kv_evict(c, w, kd, ld, od, td, fd, cd, max_seqlen_k=64, out=out)
    with pytest.raises(B.AttnError) as err:
        e.check()
    assert err.value.status == status
    assert e.seqlens.tolist() == lens and e.position_offsets.tolist() == [4, 5, 6] and e.free_count.tolist() == [count]
    assert fd.tolist() == free and td.tolist() == table
    for got, ref in ((c.k, kc), (c.v, vc), (c.k_exp, ke), (c.v_exp, ve)):
        assert torch.equal(got.view(torch.uint8).cpu(), ref)
    assert torch.equal(w.weight.cpu(), weight) and torch.equal(w.position.cpu(), position)


@pytest.mark.parametrize("layout", ["heads outside rows", "rows apart"])
def test_other_cache_layouts(B, layout):
    g, table, pool, kc, ke, vc, ve = small(B, lens=(90, 60))
    plain = handle(B, kc, vc, ke, ve)

    def lay(x):
        x = x.cuda().view(torch.float8_e4m3fn)
        if layout == "heads outside rows":
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        wide = torch.zeros((*x.shape[:3], x.shape[3] + 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        wide[..., :64].view(torch.uint8).copy_(x.view(torch.uint8))
        return wide[..., :64]

    other = B.KvCache(lay(kc), lay(vc), ke.cuda(), ve.cuda())
    weight, position = random_weights(pool, 2, 16, g)
    q, lse = torch.randn((2, 4, 64), generator=g).bfloat16().cuda(), torch.full((4, 2), 3.0, device="cuda")
    results = []
    for c in (plain, other):
        w = weights_of(B, weight, position)
        B.kv_weigh(q, lse, c, w, dev(table), dev([90, 60]), dev([0, 1, 2]), scale=0.125, max_seqlen_q=1, max_seqlen_k=96)
        B.kv_evict(c, w, dev([40, 60]), dev([90, 60]), dev([0, 0]), dev(table), dev([0] * pool), dev([0]), max_seqlen_k=96).check()
        results.append([w.weight, w.position, c.k_exp, c.v_exp] + [x.view(torch.uint8).contiguous() for x in (c.k, c.v)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_plan_with_position_offsets(B):
    for cap, batch in ((100, 3), (2000, 3)):      # one kernel, and two
        new, lens, off = [5, -1, 40], [20, 33, 0], [100, 200, 7]
        table = [[0, 1, 9, 9], [2, 3, 4, 9], [9, 9, 9, 9]]
        od = dev(off)
        p = B.kv_plan(dev(new), dev(lens), dev(table), dev([5, 6, 7, 8] + [0] * 6), dev([4]), page_size=16, max_tokens=cap,
                      position_offsets=od)
        p.check()
        assert p.positions.tolist() == [100 + 20 + i for i in range(5)] + [7 + i for i in range(40)] + [0] * (cap - 45)
        assert od.tolist() == [100, 0, 7] and p.slots[:5].tolist() == [16 * 1 + 4 + i for i in range(5)]
        bad = B.kv_plan(dev([5, -1, 400]), dev(lens), dev(table), dev([5, 6, 7, 8] + [0] * 6), dev([4]), page_size=16,
                        max_tokens=cap, position_offsets=dev(off))
        assert int(bad.status) != 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,page,d,dv", [(torch.bfloat16, 16, 128, 128), (torch.float16, 32, 64, 64)])
def test_serving_loop_with_a_budget(B, dtype, page, d, dv, graph):
    """plan, rope, append, attention, weigh and evict, step by step on the device's own
    state; each operator against the oracle, the positions against a plain count."""
    g = torch.Generator().manual_seed(d)
    batch, hkv, group, cols, cap, budget, slack, sink, recent = 3, 2, 2, 8, 160, 60, 5, 2, 10
    cols = cols * 16 // page + 6
    pool, scale = 3 * cols, d ** -0.5
    steps = [[100, 7, 0], [1, 1, 90], [1, 1, 1], [1, -1, 1], [1, 0, 1], [3, 30, 1], [1, 40, -1]] + [[1, 1, 1]] * 6
    f = B.rope_frequencies(d)
    c = handle(B, torch.zeros((pool, page, hkv, d), dtype=torch.uint8), torch.zeros((pool, page, hkv, dv), dtype=torch.uint8),
               torch.full((pool, hkv), 127, dtype=torch.uint8), torch.full((pool, hkv), 127, dtype=torch.uint8))
    w = B.KvWeights.empty(c)
    td, fd, ld, cd, od = dev([[-1] * cols] * batch), dev(list(range(pool))), dev([0] * batch), dev([pool]), dev([0] * batch)
    nd, kd = dev([0] * batch), dev([budget] * batch)
    qd = torch.zeros((cap, hkv * group, d), dtype=dtype, device="cuda")
    xd, vd = torch.zeros((cap, hkv, d), dtype=dtype, device="cuda"), torch.zeros((cap, hkv, dv), dtype=dtype, device="cuda")
    plan = B.KvPlan(torch.empty(batch + 1, dtype=I32, device="cuda"), ld, torch.empty(cap, dtype=I32, device="cuda"),
                    torch.empty(cap, dtype=torch.int64, device="cuda"), cd, dev([0]))
    gone = B.KvEviction(ld, od, cd, dev([0]))
    bounds = dict(max_seqlen_q=100, max_seqlen_k=cols * page)

    def first():
        p = B.kv_plan(nd, ld, td, fd, cd, page_size=page, max_tokens=cap, position_offsets=od, out=plan)
        rq, rk = B.rope(qd, xd, p.positions, f)
        B.kv_append(rk, vd, p.slots, c)
        o, lse = B.attn_kv_forward(rq, c, td, p.seqlens, p.cu_seqlens, scale=scale, **bounds)
        return rq, o, lse

    def second(rq, lse):
        B.kv_weigh(rq, lse, c, w, td, ld, plan.cu_seqlens, scale=scale, position_offsets=od, **bounds)

    def third():
        B.kv_evict(c, w, kd, ld, od, td, fd, cd, sink=sink, recent=recent, slack=slack, max_seqlen_k=cols * page, out=gone)

    def captured(f, *a):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            held = f(*a)
        return gr, held

    if graph:
        g1, held = captured(first)
        g2, _ = captured(second, held[0], held[2])
        g3, _ = captured(third)
    state = lambda: [x.view(torch.uint8).cpu() for x in (c.k, c.v, c.k_exp, c.v_exp)]   # noqa: E731
    seen, evictions = [0] * batch, 0
    for new in steps:
        n = sum(max(x, 0) for x in new)
        for dst in (qd, xd, vd):
            dst.copy_(torch.randn(dst.shape, generator=g).to(dtype))
        nd.copy_(torch.tensor(new, dtype=I32))
        weight, position = w.weight.cpu(), w.position.cpu()
        if graph:
            g1.replay()
            rq, o, lse = held
        else:
            rq, o, lse = first()
        plan.check()
        lens, table, cu, offsets = ld.tolist(), td.tolist(), plan.cu_seqlens.tolist(), od.tolist()
        want = []
        for b, x in enumerate(new):
            seen[b] = 0 if x < 0 else seen[b]
            want += list(range(seen[b], seen[b] + max(x, 0)))
            seen[b] += max(x, 0)
        assert plan.positions.tolist()[:n] == want                       # true positions, whatever was evicted
        assert [a + b for a, b in zip(lens, offsets)] == seen
        kc, vc, ke, ve = state()
        ref = kv_ref.attend(rq.cpu()[:n], cu, lens, table, kc, vc, ke, ve, scale, 2)
        check_attend(o[:n], lse[:, :n], ref, dtype, d, max(lens), dtype)
        g2.replay() if graph else second(rq, lse)
        w.check()
        ww, where, tol = evict_ref.weigh(rq.cpu()[:n], lse.cpu()[:, :n], cu, lens, table, kc, ke, weight, position, offsets, scale)
        assert bool(((w.weight.cpu().double() - ww).abs() <= tol).all()) and torch.equal(w.position.cpu(), where)
        for b, x in enumerate(new):                                      # what a query spreads over the keys is 1
            if x == 1 and lens[b] == 1:
                assert abs(float(w.weight[table[b][0], 0, 0]) - group) < 1e-2
        weight, position, free, count = w.weight.cpu(), w.position.cpu(), fd.tolist(), int(cd)
        g3.replay() if graph else third()
        gone.check()
        after, forgotten, left = evict_ref.evict([budget] * batch, lens, offsets, table, free, count, {"k": kc, "v": vc},
                                                 {"k": ke, "v": ve}, weight, position, sink, recent, slack)
        evictions += sum(a != b for a, b in zip(after, lens))
        assert ld.tolist() == after and od.tolist() == forgotten and cd.tolist() == [left] and fd.tolist() == free
        for got, x in zip(state(), (kc, vc, ke, ve)):
            assert torch.equal(got, x)
        assert torch.equal(w.weight.cpu(), weight) and torch.equal(w.position.cpu(), position)
    assert evictions >= 4


def test_offsets_past_32_bits(B):
    """Pages whose bytes lie more than 2^32 from the cache's first."""
    hkv, d, page, pages = 8, 256, 256, 9000
    k = torch.zeros((pages, page, hkv, d), dtype=torch.uint8, device="cuda")
    v = torch.zeros((pages, page, hkv, d), dtype=torch.uint8, device="cuda")
    e = torch.full((pages, hkv), 127, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(2)
    table = [[pages - 1, 0, pages - 2]]
    for p in table[0]:
        for x in (k, v):
            x[p] = random_cache(1, page, hkv, d, g)[0][0].cuda()
    c = B.KvCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), e, e.clone())
    w = B.KvWeights.empty(c)
    q = torch.randn((1, 16, d), generator=g).bfloat16()
    lse = torch.full((16, 1), 5.0)
    B.kv_weigh(q.cuda(), lse.cuda(), c, w, dev(table), dev([700]), dev([0, 1]), scale=1e-4, max_seqlen_q=1, max_seqlen_k=768)
    w.check()
    near = [0, 1, 2]
    kc, vc = (torch.stack([x[p].cpu() for p in table[0]]) for x in (k, v))
    ke = torch.full((3, hkv), 127, dtype=torch.uint8)
    weight, position = torch.zeros((3, hkv, page)), torch.zeros((3, hkv, page), dtype=I32)
    want, where, slack = evict_ref.weigh(q, lse, [0, 1], [700], [near], kc, ke, weight, position, [0], 1e-4)
    got = torch.stack([w.weight[p].cpu() for p in table[0]])
    assert bool(((got.double() - want).abs() <= slack).all())
    free, count = torch.zeros(pages, dtype=I32, device="cuda"), dev([0])
    B.kv_evict(c, w, dev([300]), dev([700]), dev([0]), dev(table), free, count, max_seqlen_k=768).check()
    exps = {"k": ke, "v": ke.clone()}
    where = torch.stack([torch.zeros((hkv, page), dtype=I32)] * 3)
    evict_ref.evict([300], [700], [0], [near], [0] * 3, 0, {"k": kc, "v": vc}, exps, got, where)
    for i, p in enumerate(table[0]):
        assert torch.equal(k[p].cpu(), kc[i]) and torch.equal(v[p].cpu(), vc[i])


@pytest.mark.parametrize("lens,new,bound", [
    ([150] * 3 + [900] + [40] * 300 + [333], [1] * 3 + [300] + [1] * 300 + [200], 1 << 17),   # two lists, few long segments
    ([700, 260, 500], [600, 250, 140], 1 << 16),                                             # a list, several items a CTA
])
def test_weigh_loose_bounds(B, lens, new, bound):
    """Long segments among short ones under a bound that leaves room for many: they are
    listed on the device, and their weights are those of a tight bound, but for the order
    of the additions, which the bounds decide: a rounding per query row and side."""
    g = torch.Generator().manual_seed(len(lens))
    page, hkv, group, d = 16, 2, 2, 64
    table, pool = block_table(lens, page, g)
    kc, ke = random_cache(pool, page, hkv, d, g)
    c = handle(B, kc, kc.clone(), ke, ke.clone())
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], hkv * group, d), generator=g).bfloat16()
    lse = torch.full((hkv * group, cu[-1]), 4.0)
    weight, position = random_weights(pool, hkv, page, g)
    wide = torch.zeros((len(lens), bound // page), dtype=I32)
    wide[:, :len(table[0])] = torch.tensor(table)
    results = []
    for td, most in ((dev(table), max(lens)), (wide.cuda(), bound)):
        w = weights_of(B, weight, position)
        B.kv_weigh(q.cuda(), lse.cuda(), c, w, td, dev(lens), dev(cu), scale=0.1, max_seqlen_q=max(new), max_seqlen_k=most)
        w.check()
        results.append(w)
    a, b = (w.weight.double() for w in results)
    assert bool(((a - b).abs() <= 2 * 2.0 ** -24 * (max(new) * group + 8) * b.abs()).all())
    assert torch.equal(results[0].position, results[1].position)
    if len(lens) < 10:
        want, where, slack = evict_ref.weigh(q, lse, cu, lens, table, kc, ke, weight, position, [0] * len(lens), 0.1)
        assert bool(((results[1].weight.cpu().double() - want).abs() <= slack).all())
