"""Serving operators at the edges of what their calls allow: overflowed keys,
pages that a request keeps filling, handles whose tensors moved, weights and
caches at the end of the 16-bit ranges, calls from two threads."""
import math
import subprocess
import sys
import threading

import pytest
import torch

from oracle import kv_ref
from tests.kv_cases import F64, block_table, check_attend, half_step, random_cache
from tests.test_gpu_kv import attend_case, dev, handle, runs
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------- plan

def plan_problem(batch, seed, most_new=4, room=100):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 60, (batch,), generator=g).tolist()
    new = torch.randint(-1, most_new + 1, (batch,), generator=g).tolist()
    table, pool = block_table(lens, 16, g, extra_pages=batch, extra_cols=2)
    used = {p for row in table for p in row if p >= 0}
    free = [p for p in range(pool) if p not in used]
    count = len(free)
    free += [0] * (pool - count)
    return new, lens, table, free, count, sum(max(n, 0) for n in new) + room


FIRST_PLAN = """
import sys
sys.path.insert(0, {root!r})
import torch
from head_attention_backward_gb300 import binding as B
batch, new = int(sys.argv[1]), int(sys.argv[2])
i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
lens = i(batch)
lens[:new] = 1
p = B.kv_plan(lens, i(batch), i(batch, 2), torch.arange(2 * batch, dtype=torch.int32, device="cuda"), i(1) + 2 * batch,
              page_size=16, max_tokens=new)
p.check()
assert p.cu_seqlens.tolist() == [min(b, new) for b in range(batch + 1)]
assert p.slots.tolist() == [16 * (2 * batch - 1 - t) for t in range(new)]
"""


@pytest.mark.parametrize("batch", [3047, 3048, 3071, 3073])
@pytest.mark.parametrize("tokens", [100, 3000])
def test_first_plan_of_a_process(B, batch, tokens):
    """No larger call before it has widened what the kernel may use."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_PLAN.format(root=root), str(batch), str(tokens)], capture_output=True,
                       text=True, cwd=root, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_plans_from_two_threads(B):
    """Batches of different sizes at the same time, on a stream each."""
    sizes, errors = (3100, 8192), []

    def work(batch):
        try:
            s = torch.cuda.Stream()
            new, lens, table, free, count, cap = plan_problem(batch, batch)
            want = kv_ref.plan(new, lens, [list(r) for r in table], list(free), count, 16, cap)
            with torch.cuda.stream(s):
                nd, ld, cd = dev(new), dev(lens), dev([count])
                td, fd = dev(table), dev(free)
                for _ in range(40):
                    p = B.kv_plan(nd, ld, td.clone(), fd.clone(), cd, page_size=16, max_tokens=cap)
                    p.check()
                    got = (p.cu_seqlens.tolist(), p.seqlens.tolist(), p.positions.tolist(), p.slots.tolist(),
                           p.free_count.tolist()[0])
                    assert got == tuple(want)
        except BaseException as e:   # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("page", [-1, 12, 2 ** 31 - 1])
@pytest.mark.parametrize("room", [0, 3000])
def test_plan_checks_the_page_that_a_request_fills(B, page, room):
    """New tokens in the partly filled last page: its entry has to name a page, as
    those that are pushed and popped.  A full last page, or one of a request
    without new tokens, is not written and not looked at."""
    table = [[0, 1, -1], [2, -1, -1], [3, -1, -1]]
    lens, free, count = [20, 16, 7], [4, 5, 6, 7, 8, 9, 10, 11, 0, 0, 0, 0], 8

    def run(new, rows):
        cap = sum(new) + room
        td, fd = dev(rows), dev(free)
        p = B.kv_plan(dev(new), dev(lens), td, fd, dev([count]), page_size=16, max_tokens=cap)
        return p, td, fd, cap

    bad = [list(r) for r in table]
    bad[0][1] = page
    p, td, fd, cap = run([3, 1, 0], bad)
    assert int(p.status) == B.ATTN_ERR_BAD_PAGE
    assert td.tolist() == bad and fd.tolist() == free and p.seqlens.tolist() == lens
    assert p.free_count.tolist() == [count] and p.cu_seqlens.tolist() == [0] * 4 and p.slots.tolist() == [-1] * cap
    # entries that this step has no use for
    bad[0][0], bad[1][0], bad[2][0] = page, page, page
    p, td, fd, cap = run([0, 2, 0], bad)
    p.check()
    assert p.slots.tolist() == [11 * 16, 11 * 16 + 1] + [-1] * room


def test_plan_names_the_tensor_it_refuses(B):
    i = dev([1, 1])
    td = dev([[0, -1], [1, -1]])
    with pytest.raises(ValueError, match="free_pages"):
        B.kv_plan(i, i, td, dev([[2, 3]]), dev([2]), page_size=16, max_tokens=2)
    with pytest.raises(ValueError, match="new_lens"):
        B.kv_plan(dev([[1, 1]]), i, td, dev([2, 3]), dev([2]), page_size=16, max_tokens=2)


# -------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dqk,dv,page", [(64, 64, 16), (192, 128, 32), (256, 256, 256)])
@pytest.mark.parametrize("order", ["run", "list"])
def test_append_one_infinity_leaves_the_page(B, dtype, dqk, dv, page, order):
    """An overflowed value is clamped to the largest of the scale that the finite
    ones ask for: the rows before it and its neighbours keep their values."""
    heads, pages = 2, 5
    g = torch.Generator().manual_seed(dqk)
    kc, ke = random_cache(pages, page, heads, dqk, g)
    vc, ve = random_cache(pages, page, heads, dv, g)
    slots = runs([(3, 5, 7), (0, 0, page), (2, page - 1, 1), (4, 0, 2), (1, 1, 1)], page)
    if order == "list":
        slots[1], slots[4] = slots[4], slots[1]
        slots[8], slots[9] = slots[9], slots[8]
    n = len(slots)
    k = torch.randn((n, heads, dqk), generator=g).to(dtype)
    v = torch.randn((n, heads, dv), generator=g).to(dtype)
    k[2, 0, 7], k[3, 1, dqk - 1] = math.inf, -math.inf
    v[7 + page // 2, 1, :9] = torch.tensor([math.inf, -math.inf, math.nan] * 3)
    v[7 + page, :, 3] = -math.inf
    k[7 + page + 1:7 + page + 3, 0] = math.inf           # a run of nothing finite: the least scale
    v[n - 1, 0, 1:] = 0.0
    v[n - 1, 0, 0] = math.inf
    c = handle(B, kc, vc, ke, ve)
    B.kv_append(k.cuda(), v.cuda(), dev(slots, torch.int64), c)
    kv_ref.append(kc, ke, k, slots)
    kv_ref.append(vc, ve, v, slots)
    assert int(ke[0].max()) < 127 + 5 and int(ke[3].max()) < 127 + 5
    nan = lambda x: (x & 127) == 127   # noqa: E731
    for name, got, ref in (("k", c.k, kc), ("v", c.v, vc)):
        got = got.view(torch.uint8).cpu()
        assert torch.equal(nan(got), nan(ref)) and torch.equal(got[~nan(ref)], ref[~nan(ref)]), name
    assert torch.equal(c.k_exp.cpu(), ke) and torch.equal(c.v_exp.cpu(), ve)


# ------------------------------------------------------------ tensors that move

def test_a_handle_whose_tensors_moved_is_refused(B):
    """The handle holds addresses: a tensor that was given other memory since must
    not be written through the old one."""
    def make():
        return [torch.zeros((4, 16, 2, 64), dtype=torch.uint8, device="cuda") for _ in range(2)] + [
            torch.full((4, 2), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]

    k, sl = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda"), dev([0, 1], torch.int64)
    q, td = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda"), dev([[0]])
    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=16)
    for i in range(4):
        t = make()
        c = B.KvCache(*t)
        B.kv_append(k, k, sl, c)
        B.attn_kv_forward(q, c, td, dev([2]), dev([0, 1]), **kw)
        kept = t[i].detach()                             # the old memory stays alive
        was = kept.clone()
        t[i].data = torch.zeros_like(kept)
        for _ in range(2):
            with pytest.raises(ValueError, match="moved"):
                B.kv_append(k * 3, k * 3, sl, c)
            with pytest.raises(ValueError, match="moved"):
                B.attn_kv_forward(q, c, td, dev([2]), dev([0, 1]), **kw)
            assert torch.equal(kept, was) and not bool(t[i].any())
            t[i].data = kept                             # back: the handle holds again
            B.kv_append(k, k, sl, c)
            t[i].data = torch.zeros_like(kept)
    t = make()
    with pytest.raises(ValueError, match="moved"):       # a tuple's replacement of a field
        B.kv_append(k, k, sl, B.KvCache(*t)._replace(k=torch.zeros_like(t[0])))


def test_outputs_given_by_the_caller_count_as_changed(B):
    """Autograd refuses a backward pass over a saved tensor that was overwritten
    since; it learns of it by the tensor's version."""
    pos, f = dev([1, 2]), B.rope_frequencies(64)
    x = torch.randn((2, 3, 64), device="cuda", requires_grad=True)
    y = x.exp()                                          # saves its result
    z, _ = B.rope(y, None, pos, f)
    B.rope(y, None, pos, f, out=(y.detach(), None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    q, k = torch.randn((2, 3, 64), device="cuda"), torch.randn((2, 1, 64), device="cuda")
    was = q._version, k._version
    B.rope(q, k, pos, f)
    assert (q._version, k._version) == was
    B.rope(q, k, pos, f, out=(q, k))
    assert q._version > was[0] and k._version > was[1]
    # the other calls: outputs, and what they update
    qq, table, kc, vc, ke, ve, cu = attend_case(64, 64, torch.bfloat16, 16, [5, 9], [1, 1], 1, 2)
    c, qd, td, ld, cud = handle(B, kc, vc, ke, ve), qq.cuda(), dev(table), dev([5, 9]), dev(cu)
    o, lse = torch.empty_like(qd), torch.empty((2, 2), device="cuda")

    def change(call, *tensors):
        was = [t._version for t in tensors]
        call()
        return [t._version > w for t, w in zip(tensors, was)]

    kw = dict(scale=0.1, max_seqlen_q=1, max_seqlen_k=16)
    assert change(lambda: B.attn_kv_forward(qd, c, td, ld, cud, out=(o, lse), **kw), o, lse, qd, td) == [True, True, False,
                                                                                                        False]
    kn = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    assert change(lambda: B.kv_append(kn, kn, dev([0], torch.int64), c), c.k, c.v, c.k_exp, c.v_exp, kn) == [True] * 4 + [False]
    fd, cd, nd = dev([0, 1, 2]), dev([3]), dev([1, 1])
    out = B.KvPlan(dev([0] * 3), ld, dev([0] * 2), dev([0] * 2, torch.int64), cd, dev([0]))
    td = dev([[3, -1], [4, -1]])
    assert change(lambda: B.kv_plan(nd, ld, td, fd, cd, page_size=16, max_tokens=2, out=out), td, fd, *out, nd) == [True] * 8 + [
        False]
    with torch.inference_mode():                         # tensors without a version
        i = torch.randn((2, 3, 64), device="cuda")
    want, _ = B.rope(i, None, pos, f)
    B.rope(i, None, pos, f, out=(i, None))
    assert torch.equal(i, want)


# ------------------------------------------------------------ attention's numerics

def test_weights_under_a_smaller_scale_are_rounded_once(B):
    """A light key whose page has V scales 2^4 below the accumulator's: its weight
    w in [2^-15, 2^-14) meets fp16's steps of 2^-24 and is rounded to them once,
    from fp32.  Key 0 has weight 1 and V = 0, key 64 (the same warp's next tile)
    weight w and V = 448 2^2 against 2^6; all others have none.

    The kernel's w is off by 2^-18 of itself at most (score in log2 units below
    2^4 at 2^-24, its exponential 2^-22); weights within 2^-6 of a step of a tie
    are left out (2^-6 2^-24 / 2^-15 = 2^-15).  What is left of O l / (448 2^2 2^4)
    is the rounded weight, off by half a step of O and the same 2^-18 of l."""
    n, d, page = 512, 64, 16
    g = torch.Generator().manual_seed(5)
    kc, vc = (torch.zeros((5, page, 1, d)) for _ in range(2))
    kc[:, :, :, 1] = -448.0
    kc[0, 0, 0, 1] = kc[4, 0, 0, 1] = 0.0
    kc[4, 0, 0, 0] = kc[4, 0, 0, 2] = 1.0
    vc[4, 0, 0] = 448.0
    ke = torch.full((5, 1), 127, dtype=torch.uint8)
    ve = torch.full((5, 1), 127 + 6, dtype=torch.uint8)
    ve[4] = 127 + 2
    q = torch.zeros((n, 1, d))
    q[:, 0, 0] = -(9.72 + 0.65 * torch.rand(n, generator=g))
    q[:, 0, 1] = 1.0
    q[:, 0, 2] = 0.01 * torch.rand(n, generator=g)
    q = q.half()
    f8 = torch.float8_e4m3fn
    o, _ = B.attn_kv_forward(q.cuda(), B.KvCache(kc.to(f8).cuda(), vc.to(f8).cuda(), ke.cuda(), ve.cuda()),
                             dev([[0, 1, 2, 3, 4]] * n), dev([80] * n), dev(list(range(n + 1))), scale=1.0, mask=0,
                             max_seqlen_q=1, max_seqlen_k=80, check_status=True)
    w = torch.exp(q[:, 0, 0].to(F64) + q[:, 0, 2].to(F64))
    assert bool(((w > 2.0 ** -15) & (w < 2.0 ** -14)).all())
    steps = w * 2.0 ** 24
    clear = ((steps % 1) - 0.5).abs() > 2.0 ** -6
    assert int(clear.sum()) > n // 2
    got = o[:, 0].cpu().to(F64) * (1 + w)[:, None] / (448 * 2.0 ** 2) * 2.0 ** 24
    want = torch.round(steps)
    err = (got - want[:, None]).abs().amax(1)
    lim = want * (half_step(torch.float16) + 2.0 ** -17)
    assert bool((err <= lim)[clear].all()), f"{int((err > lim)[clear].sum())} of {int(clear.sum())} rounded otherwise"


def rows_of(ref, rows):
    return tuple(x[rows] if i in (0, 2) else x[:, rows] for i, x in enumerate(ref))


@pytest.mark.parametrize("name,d,lens,new,hkv,group,scale,short", [
    ("beside a long one", 128, [30, 200, 40, 25], [1, 150, 5, 20], 2, 4, 0.01, (0, 2, 3)),
    ("head dim 256", 256, [100, 40], [90, 30], 1, 2, 0.002, (0, 1)),
    ("little work", 64, [60, 48], [48, 30], 1, 4, 0.01, (0, 1)),
    ("one head to a group", 64, [130], [120], 1, 1, 0.01, (0,)),
    ("negative scale", 64, [140], [130], 1, 2, -0.01, (0,)),
])
def test_short_segments_keep_11_bits_of_their_weights(B, name, d, lens, new, hkv, group, scale, short):
    """Segments that the tensor-core forward does not take, by the header's rule: up
    to 24 tokens, 24 + 96 / G where there is little to do, and all at head dim 256
    or a negative scale.  Many keys of like weight make O small beside sum p |v|, so
    that weights of 8 bits would leave the bounds (at 70 to 770 elements)."""
    q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.bfloat16, 16, lens, new, hkv, group, q_scale=2.0)
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=scale,
                               max_seqlen_q=max(new), max_seqlen_k=max(lens), check_status=True)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, scale, 2)
    rows = [r for b in short for r in range(cu[b], cu[b + 1])]
    check_attend(o[rows], lse[:, rows], rows_of(ref, rows), torch.bfloat16, d, max(lens), torch.float16, what=name)


def test_fp16_segments_over_tiny_scales(B):
    """Cache values below fp16's steps (scales near 2^-25).  A short segment takes
    them exactly; a long one has them rounded to multiples of 2^-24: every key and
    value is off by 2^-25 at most, a score by 2^-25 sum |q| scale =: ds."""
    lens, new, d, scale = [300, 300], [150, 4], 64, 300.0
    q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.float16, 16, lens, new, 1, 1, q_scale=30.0)
    g = torch.Generator().manual_seed(1)
    for e in (ke, ve):
        e[:] = torch.randint(127 - 30, 127 - 20, e.shape, generator=g).to(torch.uint8)
    o, lse = B.attn_kv_forward(q.cuda(), handle(B, kc, vc, ke, ve), dev(table), dev(lens), dev(cu), scale=scale,
                               max_seqlen_q=150, max_seqlen_k=300, check_status=True)
    ref = kv_ref.attend(q, cu, lens, table, kc, vc, ke, ve, scale, 2)
    short = list(range(150, 154))
    check_attend(o[short], lse[:, short], rows_of(ref, short), torch.float16, d, 300)
    rows = list(range(150))
    ro, rl, mag, size = rows_of(ref, rows)
    ds = 2.0 ** -25 * q[rows].to(F64).abs().sum(-1).T * scale + d * 2.0 ** -23 * size     # [1, T]
    rel = 2 * ds + half_step(torch.float16) + 2.0 ** -16 + 40 * 2.0 ** -24
    # weights of less than 2^-24 of the row's largest may be lost: 300 of them
    lim = rel.T[..., None] * mag + 2 * 2.0 ** -25 + half_step(torch.float16) * ro.abs() + 300 * 2.0 ** -24 * 448 * 2.0 ** -20
    assert bool(((o[rows].cpu().to(F64) - ro).abs() <= lim).all())
    assert bool(((lse[:, rows].cpu().to(F64) - rl).abs() <= ds + 2.0 ** -15 + 2.0 ** -22 * rl.abs()).all())


@pytest.mark.parametrize("keys,new", [(300, 150), (5000, 130), (90, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_scores_give_nan_in_every_path(B, keys, new, dtype):
    """A row of q with a NaN: O and LSE are NaN, not the -inf of a row that sees no
    key; its neighbours are what they were.  Long, long with split keys, short."""
    q, table, kc, vc, ke, ve, cu = attend_case(64, 64, dtype, 16, [keys], [new], 1, 1)
    args = (handle(B, kc, vc, ke, ve), dev(table), dev([keys]), dev(cu))
    kw = dict(scale=0.1, max_seqlen_q=new, max_seqlen_k=keys)
    want = B.attn_kv_forward(q.cuda(), *args, **kw)
    q[1, 0, 3] = math.nan
    o, lse = B.attn_kv_forward(q.cuda(), *args, **kw)
    assert bool(torch.isnan(o[1]).all()) and bool(torch.isnan(lse[:, 1]).all())
    others = [0] + list(range(2, new))
    assert torch.equal(o[others], want[0][others]) and torch.equal(lse[:, others], want[1][:, others])


def test_steps_from_two_threads(B):
    """Rotation, append and attention (short and long segments) of two caches at the
    same time, on a stream each: the bits of the calls made one after the other."""
    errors, jobs = [], []
    for d, lens, new in ((64, [300, 20, 90], [130, 1, 2]), (128, [2000, 5], [1, 1])):
        q, table, kc, vc, ke, ve, cu = attend_case(d, d, torch.bfloat16, 16, lens, new, 2, 4)
        slots = [table[b][i // 16] * 16 + i % 16 for b, n in enumerate(lens) for i in range(n - new[b], n)]
        pos = [i for b, n in enumerate(lens) for i in range(n - new[b], n)]
        k, v = torch.randn_like(q[:, :2]).cuda(), torch.randn_like(q[:, :2]).cuda()
        jobs.append((B.rope_frequencies(d), q.cuda(), k, v, dev(pos), dev(slots, torch.int64), dev(table), dev(lens), dev(cu),
                     (kc, vc, ke, ve), dict(scale=0.1, max_seqlen_q=max(new), max_seqlen_k=max(lens))))

    def step(job):
        f, q, k, v, pos, slots, table, lens, cu, cache, kw = job
        c = handle(B, *cache)
        rq, rk = B.rope(q, k, pos, f)
        B.kv_append(rk, v, slots, c)
        o, lse = B.attn_kv_forward(rq, c, table, lens, cu, **kw)
        return [x.cpu() for x in (o, lse, c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_exp, c.v_exp)]

    def work(job, want):
        try:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(s):
                for _ in range(30):
                    for a, b in zip(step(job), want):
                        assert torch.equal(a, b)
        except BaseException as e:   # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j, step(j))) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
