"""Attention weights of many long segments in one call on the GPU: more 128-key items than
CTAs, so that each CTA takes several, one after another, in the same shared memory,
barriers and TMEM.  Against sums of exp(score - LSE) in 64 bits."""
import math

import pytest
import torch

from oracle import attn_ref, kv_ref
from tests.kv_cases import block_table, random_cache
from tests.test_gpu_evict import random_weights, weigh_case, weights_of
from tests.test_gpu_kv import dev, handle
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

I32, F64 = torch.int32, torch.float64
MOST_CTAS = 608     # of the long segments' kernel where its items are listed
KEYS = 128          # of an item


def weighed(q, lse, cu, lens, table, kc, ke, weight, position, scale, mask, left, right, decay):
    """New weights and positions, and how far a kernel's may be off: per probability p its
    score's error (d products in fp32 accumulators, 2^-23 of the sum of their magnitudes)
    and the exponent's argument and ex2 (2^-22 (|s| + |LSE| + 1)), and a rounding per
    addition, 2^-23 of the sum."""
    page, group = kc.shape[1], q.shape[1] // kc.shape[2]
    out, where, slack = weight.to(F64).clone(), position.clone(), torch.zeros(weight.shape, dtype=F64)
    for b, n in enumerate(lens):
        lq = cu[b + 1] - cu[b]
        if lq == 0 or n == 0:
            continue
        see = attn_ref.visible(lq, n, mask, left, right)
        k = kv_ref.gather(kc, ke, table[b][: (n + page - 1) // page], n).to(F64)
        j = torch.arange(n)
        at = (torch.tensor(table[b])[j // page], slice(None), j % page)          # -> [n, heads]
        fresh = j >= n - lq
        qs = q[cu[b]:cu[b + 1]].to(F64).unflatten(1, (-1, group))
        ls = lse[:, cu[b]:cu[b + 1]].to(F64).unflatten(0, (-1, group))[..., None]
        s = torch.einsum("qhgd,khd->hgqk", qs, k) * scale
        size = torch.einsum("qhgd,khd->hgqk", qs.abs(), k.abs()) * abs(scale)
        p = torch.where(see, torch.exp(s - ls), torch.zeros_like(s))
        err = p * (q.shape[2] * 2.0 ** -23 * size + 2.0 ** -22 * (s.abs() + ls.abs() + 1))
        got, err = p.sum((1, 2)).T, err.sum((1, 2)).T
        old = torch.where(fresh[:, None] | (decay == 0.0), torch.zeros_like(got), decay * out[at])
        touched = (see.any(0) | fresh | (decay != 1.0))[:, None]
        out[at] = torch.where(touched, old + got, out[at])
        slack[at] = torch.where(touched, err + 2.0 ** -23 * (lq * group + 8) * (old.abs() + got), torch.zeros_like(got))
        where[at] = torch.where(fresh[:, None], j.to(I32)[:, None], where[at])
    return out, where, slack


MANY = [
    # segments, of which long, kv heads, group, d, d_v, mask, left, decay
    (64, 64, 8, 3, 64, 64, 2, -1, 1.0), (64, 64, 8, 3, 128, 128, 2, -1, 0.5),          # rows of a tile that no head fills
    (70, 70, 8, 1, 192, 128, 2, -1, 1.0), (64, 64, 8, 5, 256, 256, 2, -1, 1.0),
    (64, 64, 8, 3, 128, 128, 3, 40, 0.75),                                           # items that no query sees: decay alone
    (530, 90, 8, 2, 64, 64, 2, -1, 1.0), (300, 60, 8, 4, 128, 128, 3, 60, 0.75),         # two lists and three
]


@pytest.mark.gpu
@pytest.mark.parametrize("batch,long,hkv,group,d,dv,mask,left,decay", MANY)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weigh_several_items_a_cta(B, batch, long, hkv, group, d, dv, mask, left, decay, dtype):
    g = torch.Generator().manual_seed(batch + d)
    page = 16
    every = batch / long
    is_long = {int(i * every) for i in range(long)}
    base = 128 // group + 1                                     # the least of a long segment
    new = [base + 17 * b % 90 if b in is_long else b % 3 for b in range(batch)]
    lens = [n + 290 + 37 * b % 200 if b in is_long else n + 10 + b % 50 for b, n in enumerate(new)]
    right = 0 if mask == 3 else -1
    bound = 2048                                                # loose: the items are listed
    assert batch * hkv * (bound // KEYS + 1) > 4096
    first = [max(0, n - lq - left) if mask == 3 and decay == 1.0 else 0 for n, lq in zip(lens, new)]
    items = hkv * sum((n - 1) // KEYS - f // KEYS + 1 for b, (n, f) in enumerate(zip(lens, first)) if b in is_long)
    assert items >= 2 * MOST_CTAS
    table, pool = block_table(lens, page, g)
    kc, ke = random_cache(pool, page, hkv, d, g)
    vc, ve = random_cache(1, page, hkv, dv, g)
    c = handle(B, kc, vc.expand(pool, -1, -1, -1).contiguous(), ke, ve.expand(pool, -1).contiguous())
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], hkv * group, d), generator=g).to(dtype)
    lse = 5 + torch.randn((hkv * group, cu[-1]), generator=g)
    weight, position = random_weights(pool, hkv, page, g)
    wide = torch.full((batch, bound // page), -1, dtype=I32)
    wide[:, :len(table[0])] = torch.tensor(table)
    args = (q.cuda(), lse.cuda(), c), (wide.cuda(), dev(lens), dev(cu))
    kw = dict(scale=d ** -0.5, mask=mask, left=left, right=right, decay=decay, max_seqlen_q=max(new), max_seqlen_k=bound)
    w = weights_of(B, weight, position)
    B.kv_weigh(*args[0], w, *args[1], **kw)
    w.check()
    want, where, slack = weighed(q, lse, cu, lens, table, kc, ke, weight, position, d ** -0.5, mask, left, right, decay)
    assert torch.equal(w.position.cpu(), where)
    far = (w.weight.cpu().to(F64) - want).abs()
    assert bool((far <= slack).all()), f"{int((far > slack).sum())} weights off, by up to {float(far.max())}"
    for _ in range(3):
        again = weights_of(B, weight, position)
        B.kv_weigh(*args[0], again, *args[1], **kw)
        assert torch.equal(again.weight, w.weight)


def test_plain_form_is_the_oracles():
    """The sums above and the oracle's, on one small call."""
    from oracle import evict_ref
    g = torch.Generator().manual_seed(4)
    lens, cu = [40, 9, 0, 33], [0, 5, 5, 7, 10]
    table, pool = block_table(lens, 16, g)
    kc, ke = random_cache(pool, 16, 2, 64, g)
    q, lse = torch.randn((10, 6, 64), generator=g).bfloat16(), 4 + torch.randn((6, 10), generator=g)
    weight, position = random_weights(pool, 2, 16, g)
    for mask, left, right, decay in ((2, -1, -1, 1.0), (3, 4, 0, 1.0), (3, 4, 0, 0.5), (2, -1, -1, 0.0)):
        a = weighed(q, lse, cu, lens, table, kc, ke, weight, position, 0.1, mask, left, right, decay)
        b = evict_ref.weigh(q, lse, cu, lens, table, kc, ke, weight, position, [0] * 4, 0.1, mask, left, right, decay)
        assert torch.equal(a[1], b[1])
        assert bool(((a[0] - b[0]).abs() <= 1e-12 * (1 + b[0].abs())).all())
        assert bool(((a[2] - b[2]).abs() <= 1e-12 * (1 + b[2])).all()) and math.isfinite(float(a[2].sum()))


@pytest.mark.gpu
def test_long_segments_wait_is_bounded(B):
    """The wait of the long segments' kernel on a barrier that nobody completes gives up
    within its bound, and at once where another warp has given up before."""
    scratch = torch.zeros(B.SELFTEST_SCRATCH_BYTES, dtype=torch.uint8, device="cuda")
    rc, status = B.attn_selftest_waits(scratch.data_ptr(), scratch.numel(), torch.cuda.current_stream().cuda_stream)
    assert (rc, status) == (0, [B.ATTN_ERR_TIMEOUT, B.ATTN_ERR_TIMEOUT, 0])
    assert scratch.view(I32)[385:387].tolist() == [B.ATTN_ERR_TIMEOUT, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,hkv,group,d,dv", [([150, 40], [60, 5], 1, 130, 64, 64), ([90], [33], 2, 65, 192, 128),
                                                     ([200], [20], 1, 256, 128, 128), ([50, 20], [40, 20], 1, 80, 256, 256)])
@pytest.mark.parametrize("dtype,decay", [(torch.bfloat16, 1.0), (torch.float16, 0.5)])
def test_weigh_prompts_of_large_groups(B, lens, new, hkv, group, d, dv, dtype, decay):
    """More query heads per kv head than the long segments' kernel takes: 128 rows at a time."""
    weigh_case(B, dtype, lens, new, 16, hkv, group, d, dv, decay=decay)


@pytest.mark.gpu
def test_weigh_beside_other_calls(B):
    """Long segments of two requests at a time on two streams, a forward pass on a third:
    all of them hold TMEM; the weights are those of the calls alone."""
    g = torch.Generator().manual_seed(9)
    page, hkv, group, d, lens, new = 16, 4, 4, 128, [1500, 700], [300, 200]
    table, pool = block_table(lens, page, g)
    kc, ke = random_cache(pool, page, hkv, d, g)
    c = handle(B, kc, kc.clone(), ke, ke.clone())
    q = torch.randn((sum(new), hkv * group, d), generator=g).bfloat16().cuda()
    lse = (5 + torch.randn((hkv * group, sum(new)), generator=g)).cuda()
    weight, position = random_weights(pool, hkv, page, g)
    td, ld, cu = dev(table), dev(lens), dev([0, 300, 500])
    x, k = (torch.randn((2, 1024, h, d), generator=g).bfloat16().cuda() for h in (16, 4))
    weigh = lambda w: B.kv_weigh(q, lse, c, w, td, ld, cu, scale=0.08, max_seqlen_q=300, max_seqlen_k=1500)   # noqa: E731
    forward = lambda: B.attn_forward(x, k, k, scale=0.08, mask=1)   # noqa: E731
    one = weights_of(B, weight, position)
    weigh(one)
    o, l = forward()
    both = [[weights_of(B, weight, position) for _ in range(8)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for i in range(8):
        for s, ws in zip(streams, both):
            with torch.cuda.stream(s):
                weigh(ws[i])
        with torch.cuda.stream(streams[2]):
            outs.append(forward())
    torch.cuda.synchronize()
    for w in both[0] + both[1]:
        w.check()
        assert torch.equal(w.weight, one.weight) and torch.equal(w.position, one.position)
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, l)
