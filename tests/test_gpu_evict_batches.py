"""Eviction from large batches on the GPU: the checks of a call are shared by CTAs of 16
requests each, and a request's place on the stack of free pages counts what those before
it give back, over more requests than one CTA has threads.  Against the oracle, byte by
byte, and refused calls against their inputs."""
import pytest
import torch

from oracle import evict_ref
from tests.kv_cases import block_table, random_cache
from tests.test_gpu_evict import random_weights, weights_of
from tests.test_gpu_kv import dev, handle
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

I32 = torch.int32
PAGE = 16
# max_seqlen_k: up to 8,192 a CTA owns a request and head, beyond that a cluster does
BOUNDS = [600, 8208]


def batch_of(B, batch, seed=0):
    """Requests of up to 70 tokens, some over their budget, some without one, some empty."""
    g = torch.Generator().manual_seed(batch + seed)
    lens = torch.randint(0, 71, (batch,), generator=g).tolist()
    keep = [(-1, 0, 1, 16, 17, 30, 69)[i] for i in torch.randint(0, 7, (batch,), generator=g).tolist()]
    lens[-1], keep[-1] = 60, 20                     # the last one shrinks, and one in the middle
    lens[batch // 2], keep[batch // 2] = 55, 8
    table, pool = block_table(lens, PAGE, g, extra_pages=3)
    kc, ke = random_cache(pool, PAGE, 1, 64, g)
    vc, ve = random_cache(pool, PAGE, 1, 64, g)
    weight, position = random_weights(pool, 1, PAGE, g)
    offsets = torch.randint(0, 50, (batch,), generator=g).tolist()
    used = {p for r in table for p in r if p >= 0}
    free = [p for p in range(pool) if p not in used]
    return lens, keep, table, pool, kc, ke, vc, ve, weight, position, offsets, free


def wide(table, bound):
    t = torch.full((len(table), bound // PAGE + 1), -1, dtype=I32)
    t[:, :len(table[0])] = torch.tensor(table)
    return t


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("batch", [16, 17, 33, 513, 1100])
def test_evict_large_batches(B, batch, bound):
    lens, keep, table, pool, kc, ke, vc, ve, weight, position, offsets, free = batch_of(B, batch)
    count = len(free)
    free += [-5] * (pool - count)
    c, w, fd = handle(B, kc, vc, ke, ve), weights_of(B, weight, position), dev(free)
    td = wide(table, bound).cuda()
    e = B.kv_evict(c, w, dev(keep), dev(lens), dev(offsets), td, fd, dev([count]), sink=2, recent=9, max_seqlen_k=bound)
    e.check()
    cache, exps = {"k": kc, "v": vc}, {"k": ke, "v": ve}
    after, gone, left = evict_ref.evict(keep, lens, offsets, table, free, count, cache, exps, weight, position, 2, 9)
    assert sum(a != b for a, b in zip(after, lens)) > batch // 4
    assert e.seqlens.tolist() == after and e.position_offsets.tolist() == gone and e.free_count.tolist() == [left]
    assert fd.tolist() == free and torch.equal(td.cpu(), wide(table, bound))
    for got, ref in ((c.k, kc), (c.v, vc), (c.k_exp, ke), (c.v_exp, ve)):
        assert torch.equal(got.view(torch.uint8).cpu(), ref)
    assert torch.equal(w.weight.cpu(), weight) and torch.equal(w.position.cpu(), position)


def test_evict_the_largest_batch(B):
    """ATTN_KV_MAX_BATCH requests of one page and a token each, all of which give one back."""
    batch = 8192
    order = torch.randperm(2 * batch, generator=torch.Generator().manual_seed(1)).to(I32).view(batch, 2)
    kc = torch.zeros((2 * batch, PAGE, 1, 64), dtype=torch.uint8)
    ke = torch.full((2 * batch, 1), 127, dtype=torch.uint8)
    c = handle(B, kc, kc.clone(), ke, ke.clone())
    w = B.KvWeights.empty(c)
    free = torch.full((2 * batch,), -1, dtype=I32, device="cuda")
    e = B.kv_evict(c, w, dev([16] * batch), dev([17] * batch), dev([0] * batch), order.cuda(), free, dev([0]), max_seqlen_k=32)
    e.check()
    assert e.free_count.tolist() == [batch] and torch.equal(free[:batch].cpu(), order[:, 1])
    assert bool((free[batch:] == -1).all()) and bool((e.seqlens == 16).all()) and bool((e.position_offsets == 1).all())


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("batch", [17, 33, 1100])
@pytest.mark.parametrize("what", ["page of the last", "page of one in the middle", "length of the last", "keep of the last",
                                  "stack too full"])
def test_evict_refused_large_batches_change_nothing(B, batch, bound, what):
    lens, keep, table, pool, kc, ke, vc, ve, weight, position, offsets, free = batch_of(B, batch, seed=1)
    count, status = len(free), B.ATTN_ERR_BAD_SEQLENS
    if what == "page of the last":
        table[-1][1], status = pool, B.ATTN_ERR_BAD_PAGE
    elif what == "page of one in the middle":
        table[batch // 2][3], status = -1, B.ATTN_ERR_BAD_PAGE
    elif what == "length of the last":
        lens[-1] = 1 << 20
    elif what == "keep of the last":
        keep[-1] = -2
    else:
        after = [k if 0 <= k < n else n for n, k in zip(lens, keep)]
        back = sum((n + PAGE - 1) // PAGE - (a + PAGE - 1) // PAGE for n, a in zip(lens, after))
        count = pool - back + 1
    free = list(range(100, 100 + pool))
    c, w, fd, td = handle(B, kc, vc, ke, ve), weights_of(B, weight, position), dev(free), wide(table, bound).cuda()
    e = B.kv_evict(c, w, dev(keep), dev(lens), dev(offsets), td, fd, dev([count]), max_seqlen_k=bound)
    with pytest.raises(B.AttnError) as err:
        e.check()
    assert err.value.status == status
    assert e.seqlens.tolist() == lens and e.position_offsets.tolist() == offsets and e.free_count.tolist() == [count]
    assert fd.tolist() == free and torch.equal(td.cpu(), wide(table, bound))
    for got, ref in ((c.k, kc), (c.v, vc), (c.k_exp, ke), (c.v_exp, ve)):
        assert torch.equal(got.view(torch.uint8).cpu(), ref)
    assert torch.equal(w.weight.cpu(), weight) and torch.equal(w.position.cpu(), position)
