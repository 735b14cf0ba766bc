"""attn_rope against the fp64 oracle: types, pairings, axes, layouts, far
positions, the inverse as the gradient, and the rotation around the attention's
forward and backward pass."""
import math

import pytest
import torch

from oracle import attn_ref, kv_ref
from tests.kv_cases import F64, half_step
from tests.parity import assert_all_ok, compare
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def check(got, x, ref):
    """cos and sin carry at most 2.5e-7 (an angle below pi / 4 held in fp32,
    three roundings, and the series), the products and their sum 1.8e-7 of
    |a| + |b|; 5e-7 of the row's largest pair sum covers both.  Then one
    rounding to the output type."""
    lim = 5e-7 * 2 * x.to(F64).abs().amax(-1, keepdim=True) + half_step(x.dtype) * ref.abs()
    if x.dtype == torch.float16:
        lim = lim + 2.0 ** -25
    err = (got.cpu().to(F64) - ref).abs()
    assert bool((err <= lim).all()), f"off by {float(err.max())}"


CASES = [
    # rows, hq, hkv, d, rot, axes, dtype, interleaved, far
    (1, 1, 0, 2, 2, 1, torch.float32, False, 10),
    (1, 4, 1, 64, 64, 1, torch.bfloat16, False, 1),
    (7, 3, 1, 128, 128, 3, torch.bfloat16, False, 1 << 20),
    (33, 8, 2, 128, 64, 4, torch.float16, True, 1 << 20),
    (65, 5, 5, 64, 30, 2, torch.float16, False, 4097),
    (17, 2, 1, 192, 186, 3, torch.bfloat16, True, 999),
    (130, 4, 2, 256, 256, 1, torch.float16, False, 70000),
    (9, 2, 3, 30, 14, 2, torch.float32, False, 1 << 30),
    (40, 2, 2, 20, 20, 2, torch.float32, True, 100),
    (3, 2, 2, 32, 32, 1, torch.float32, True, 100),
    (70, 3, 2, 7, 4, 2, torch.float32, True, 100),
    (70, 3, 2, 9, 6, 2, torch.float32, False, 100),
    (3000, 9, 1, 64, 58, 2, torch.bfloat16, True, 100),
    (2500, 3, 2, 128, 96, 2, torch.float16, False, 100),
    (9001, 2, 1, 64, 64, 3, torch.bfloat16, False, 9001),
    # halves that start inside a 16-byte vector, rows of an odd number of vectors
    (700, 5, 2, 256, 250, 2, torch.float32, False, 5000),
    (1600, 3, 1, 256, 254, 1, torch.float16, False, 5000),
    (5, 1, 0, 200, 122, 3, torch.bfloat16, False, 1 << 20),
    (8100, 1, 1, 8, 2, 1, torch.bfloat16, False, 100),
    (611, 7, 3, 72, 20, 2, torch.float16, True, 100),
    (2100, 11, 2, 132, 132, 1, torch.float32, True, 100),
    (13, 4, 4, 4, 2, 1, torch.float32, False, 100),
]


@pytest.mark.parametrize("rows,hq,hkv,d,rot,axes,dtype,inter,far", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(B, rows, hq, hkv, d, rot, axes, dtype, inter, far, inverse):
    g = torch.Generator().manual_seed(rows + d)
    q = torch.randn((rows, hq, d), generator=g).to(dtype)
    k = torch.randn((rows, hkv, d), generator=g).to(dtype) if hkv else None
    pos = torch.randint(-far, far, (axes, rows), generator=g, dtype=torch.int32)
    pos[:, 0] = far
    f = B.rope_frequencies(rot)
    axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.uint8)
    qo, ko = B.rope(q.cuda(), None if k is None else k.cuda(), pos.cuda(), f, pair_axis=axis, interleaved=inter,
                    inverse=inverse)
    for x, got in ((q, qo), (k, ko)):
        if x is not None:
            ref = kv_ref.rope(x, pos, f, axis, inter, inverse)
            check(got, x, ref)
            if rot < d:
                assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["bshd", "bhsd", "sbhd", "packed", "shared_pos", "in_place"])
def test_layouts(B, dtype, layout):
    b, s, hq, hkv, d = 3, 21, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    q, k = torch.randn((b, s, hq, d), generator=g).to(dtype), torch.randn((b, s, hkv, d), generator=g).to(dtype)
    pos = torch.randint(0, 500, (2, b, s), generator=g, dtype=torch.int32)
    if layout == "shared_pos":
        pos = pos[:, :1].expand(2, b, s)
    f, axis = B.rope_frequencies(d, 500.0), (torch.arange(d // 2) % 2).to(torch.uint8)
    qd, kd = q.cuda(), k.cuda()
    if layout == "bhsd":
        qd, kd = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (qd, kd))
    elif layout == "sbhd":
        qd, kd = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (qd, kd))
    elif layout == "packed":
        both = torch.cat((qd, kd), 2)
        qd, kd = both[:, :, :hq], both[:, :, hq:]
    pd = pos.cuda() if layout != "shared_pos" else pos[:, :1].cuda().expand(2, b, s)
    out = (qd, kd) if layout in ("in_place", "packed") else None
    qo, ko = B.rope(qd, kd, pd, f, pair_axis=axis, out=out)
    if out is not None:
        assert qo is qd and ko is kd
    flat = pos.reshape(2, b * s)
    for x, got in ((q, qo), (k, ko)):
        ref = kv_ref.rope(x.reshape(b * s, -1, d), flat, f, axis).view(x.shape)
        check(got, x, ref)


def test_many_rows_in_batches(B):
    """Enough rows for eight to a CTA, heads outside the rows, a ragged last CTA,
    negative and zero frequencies."""
    b, s, hq, hkv, d = 3, 701, 3, 1, 64
    g = torch.Generator().manual_seed(8)
    q, k = torch.randn((b, s, hq, d), generator=g), torch.randn((b, s, hkv, d), generator=g)
    f = B.rope_frequencies(d)
    f[3], f[5] = -0.37, 0.0
    for dtype in (torch.bfloat16, torch.float32):
        pos = torch.randint(0, 9000, (2, b, s), generator=g, dtype=torch.int32)
        axis = (torch.arange(d // 2) % 2).to(torch.uint8)
        qq, kk = q.to(dtype), k.to(dtype)
        qd = qq.cuda().transpose(1, 2).contiguous().transpose(1, 2)
        qo, ko = B.rope(qd, kk.cuda(), pos.cuda(), f, pair_axis=axis)
        flat = pos.reshape(2, -1)
        for x, got in ((qq, qo), (kk, ko)):
            check(got, x, kv_ref.rope(x.reshape(b * s, -1, d), flat, f, axis).view(x.shape))


def test_copied_columns_keep_their_bits(B):
    """Columns past rot_dim: NaN payloads, infinities and negative zero come through."""
    x = torch.tensor([0x7fc1, 0xff80, 0x8000, 0x7f80, 1, 0xffff, 0, 0x3f80] * 8, dtype=torch.int32).to(torch.int16)
    x = x.view(torch.bfloat16).view(1, 1, 64).cuda()
    for rot, inter in ((32, False), (16, True), (6, False), (6, True)):
        y, _ = B.rope(x, None, torch.tensor([3], dtype=torch.int32, device="cuda"), B.rope_frequencies(rot),
                      interleaved=inter)
        assert torch.equal(y[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16))


def test_no_rows_and_other_stream(B):
    f = B.rope_frequencies(64)
    z = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    y, _ = B.rope(z, None, torch.empty((0,), dtype=torch.int32, device="cuda"), f)
    assert y.shape == z.shape
    q = torch.randn((50, 2, 64), device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want, _ = B.rope(q, None, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = B.rope(q, None, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_inverse_is_the_gradient(B):
    """<g, rope(x)> differentiated by central differences along random
    directions equals <rope^-1(g), direction> (rope is linear, so the
    difference quotient is exact up to fp32 rounding: 2^-24 per term times the
    root of 4096 terms, 64 times over)."""
    gen = torch.Generator().manual_seed(1)
    rows, h, d = 32, 2, 64
    x, gy, dx = (torch.randn((rows, h, d), generator=gen).cuda() for _ in range(3))
    pos = torch.randint(0, 1000, (3, rows), generator=gen, dtype=torch.int32).cuda()
    f, axis = B.rope_frequencies(48), (torch.arange(24) % 3).to(torch.uint8)
    run = lambda t, inv=False: B.rope(t, None, pos, f, pair_axis=axis, inverse=inv)[0].to(F64)   # noqa: E731
    diff = ((run(x + dx) - run(x - dx)) / 2 * gy.to(F64)).sum()
    grad = (run(gy, True) * dx.to(F64)).sum()
    assert abs(float(diff - grad)) <= 64 * 2.0 ** -24 * math.sqrt(rows * h * d) * 4
    assert float((run(run(x).float(), True) - x.to(F64)).abs().max()) <= 4e-6   # 8 roundings of values below 5


def test_around_attention(B):
    """Training: rope, forward, backward, inverse rope, against the fp64 oracle
    (its dQ and dK rotated back in 64 bits)."""
    b, s, hq, hkv, d = 2, 150, 4, 2, 64
    gen = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn((b, s, h, d), generator=gen).to(torch.bfloat16) for h in (hq, hkv, hkv, hq))
    pos = torch.stack([torch.arange(s, dtype=torch.int32).expand(b, s), torch.randint(0, 40, (b, s), generator=gen,
                                                                                      dtype=torch.int32)])
    f, axis, scale = B.rope_frequencies(d), (torch.arange(d // 2) % 2).to(torch.uint8), d ** -0.5
    pd = pos.cuda()
    rq, rk = B.rope(q.cuda(), k.cuda(), pd, f, pair_axis=axis)
    o, lse = B.attn_forward(rq, rk, v.cuda(), scale=scale, mask=B.MASK_CAUSAL_TOP_LEFT)
    dq, dk, dv = B.attn_backward(rq, rk, v.cuda(), o, do.cuda(), lse, scale=scale, mask=B.MASK_CAUSAL_TOP_LEFT,
                                 deterministic=True)
    gq, gk = B.rope(dq, dk, pd, f, pair_axis=axis, inverse=True)
    turn = lambda x, inv=False: kv_ref.rope(x.reshape(b * s, -1, d), pos.reshape(2, -1), f, axis,   # noqa: E731
                                            inverse=inv).view(x.shape)
    q64, k64 = turn(q), turn(k)
    o64, lse64 = attn_ref.attn_forward(q64, k64, v, scale, mask=1)
    ref = attn_ref.attn_backward(q64, k64, v, o64, do, lse64, scale, mask=1)
    reps = []
    for n, got, r in (("dq", gq, turn(ref[0], True)), ("dk", gk, turn(ref[1], True)), ("dv", dv, ref[2])):
        rep = compare(got.cpu(), r, 2e-2, 0.9999)
        rep["tensor"] = n
        reps.append(rep)
    assert_all_ok(reps, "rope around attention")


@pytest.mark.parametrize("dtype,d,rot,inter", [(torch.bfloat16, 128, 126, False), (torch.float32, 256, 36, False),
                                               (torch.float16, 40, 10, True), (torch.float32, 68, 68, True)])
def test_rope_staged_in_place(B, dtype, d, rot, inter):
    """Slices of a packed projection with halves that start inside a vector, rotated
    where they are: the same bits as out of place, and the rest untouched."""
    g = torch.Generator().manual_seed(d)
    qkv = torch.randn((2, 333, 9, d), generator=g).to(dtype).cuda()
    was = qkv.clone()
    pos = torch.randint(0, 9000, (2, 333), generator=g, dtype=torch.int32).cuda()
    q, k = qkv[:, :, :5], qkv[:, :, 5:7]
    f = B.rope_frequencies(rot)
    want = B.rope(q, k, pos, f, interleaved=inter)
    B.rope(q, k, pos, f, interleaved=inter, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 7:], was[:, :, 7:])
    assert not torch.equal(q, was[:, :, :5])
    back = B.rope(q, k, pos, f, interleaved=inter, inverse=True)
    # |x| < 5.5, turned below 8: half a step of each component, turned back (8 eps), the
    # last rounding (3 eps), and cos^2 + sin^2 within 3 eps of 1 (17 eps)
    assert float((back[0].double() - was[:, :, :5].double()).abs().max()) <= 28 * torch.finfo(dtype).eps
