"""8-bit activation checkpoints on the GPU: the numbers against the fp64 oracle
(equal), the backward against attn_backward at the values they stand for (the
same bits), against the oracle's gradients and against differences."""
import math

import pytest
import torch

from oracle import attn_ref as R
from oracle import ckpt_ref
from tests.parity import assert_all_ok, call_scale, compare, tolerances
from tests.test_gpu_parity import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

F64 = torch.float64
NAMES = ("q", "k", "v", "o")


def randoms(shapes, dtype, seed, spread=12):
    g = torch.Generator().manual_seed(seed)
    out = []
    for s in shapes:
        x = torch.randn(s, generator=g) * torch.exp2(torch.randint(-spread, spread // 2, (*s[:-1], 1), generator=g).float())
        x[..., 0] *= 8
        out.append(x.to(dtype))
    return out


def shapes_of(lead_q, lead_k, hq, hkv, dqk, dv):
    return [(*lead_q, hq, dqk), (*lead_k, hkv, dqk), (*lead_k, hkv, dv), (*lead_q, hq, dv)]


def check_numbers(c, xs):
    for n, x in zip(NAMES, xs):
        want, byte = ckpt_ref.quantise(x)
        assert torch.equal(getattr(c, n + "_exp").cpu(), byte), n
        assert torch.equal(getattr(c, n).cpu(), want), n


SAVES = [
    # rows of q, rows of k, heads, head dims
    ((1,), (1,), 1, 1, 64, 64), ((3, 5), (3, 7), 4, 2, 64, 64), ((130,), (257,), 6, 3, 128, 128),
    ((2, 77), (2, 33), 4, 1, 192, 128), ((1, 300), (1, 41), 2, 2, 256, 256), ((5,), (5,), 3, 1, 32, 96),
]


@pytest.mark.parametrize("lead_q,lead_k,hq,hkv,dqk,dv", SAVES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_numbers_are_the_oracles(B, lead_q, lead_k, hq, hkv, dqk, dv, dtype):
    xs = randoms(shapes_of(lead_q, lead_k, hq, hkv, dqk, dv), dtype, hq + dqk)
    c = B.checkpoint(*(x.cuda() for x in xs))
    check_numbers(c, xs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_ends_of_the_range(B, dtype):
    """Zeros, the least and largest numbers, ties, infinities and NaN, and amax on either side of 127 steps."""
    f = torch.finfo(dtype)
    x = torch.zeros((16, 2, 64), dtype=dtype)
    x[1, 0, 3] = f.max
    x[1, 1, 40] = -f.max
    x[2, 0, 5] = f.tiny
    x[2, 1, :8] = f.smallest_normal if hasattr(f, "smallest_normal") else f.tiny
    x[3, 0, 0], x[3, 0, 1:9] = 127.0, torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 63.25, -126.5]).to(dtype)
    x[4, 0, 0] = 127.5 if dtype != torch.bfloat16 else 128.0
    x[5, 0, 1] = math.inf
    x[5, 1, 33] = -math.inf
    x[6, 0, 63] = math.nan
    x[7, 0, 31], x[7, 0, 32] = 1.0, 1000.0
    if dtype == torch.float32:
        x[8, 0, 0] = 1e-40
        x[9, 0, 0], x[9, 0, 1] = 2.0 ** -120, 2.0 ** -127
    c = B.checkpoint(*(x.cuda() for _ in range(4)))
    check_numbers(c, [x] * 4)


LAYOUTS = ["BHSD", "SBHD", "packed qkv", "rows apart", "HSBD"]


def laid_out(x, layout, d):
    """x's values in another memory order, with gaps for two of them."""
    if layout == "BHSD":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "SBHD":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "HSBD":
        return x.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    if layout == "packed qkv":
        wide = torch.zeros((*x.shape[:2], 3 * x.shape[2], d), dtype=x.dtype, device=x.device)
        wide[:, :, x.shape[2]:2 * x.shape[2]] = x
        return wide[:, :, x.shape[2]:2 * x.shape[2]]
    wide = torch.zeros((x.shape[0], x.shape[1] + 3, x.shape[2], d + 8), dtype=x.dtype, device=x.device)
    wide[:, 1:-2, :, :d] = x
    return wide[:, 1:-2, :, :d]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_inputs(B, layout, dtype):
    xs = randoms(shapes_of((3, 37), (3, 20), 4, 2, 64, 64), dtype, 7)
    c = B.checkpoint(*(laid_out(x.cuda(), layout, 64) for x in xs))
    check_numbers(c, xs)
    if layout in ("BHSD", "SBHD"):        # the memory order is kept
        want = laid_out(xs[0], layout, 64).stride()
        assert c.q.stride() == want and [4 * s for s in c.q_exp.stride()[:3]] == [s // 8 for s in want[:3]]


def test_written_into_given_tensors(B):
    xs = [x.cuda() for x in randoms(shapes_of((50,), (60,), 4, 2, 128, 128), torch.bfloat16, 3)]
    c = B.checkpoint(*xs)
    d = B.AttnCheckpoint(*(torch.empty_like(x) for x in c))
    before = d.q._version
    assert B.checkpoint(*xs, out=d) is d and d.q._version > before
    for a, b in zip(c, d):
        assert torch.equal(a, b)


def test_refused_tensors(B):
    q, k, v, o = (x.cuda() for x in randoms(shapes_of((2, 9), (2, 9), 4, 2, 64, 64), torch.bfloat16, 3))
    for bad in ((q, k, v, o.float()), (q, k[:, :5], v, o), (q, k, v, o[:, :, :2]), (q[0], k, v, o), (q.cpu(), k, v, o),
                (q.transpose(2, 3), k, v, o), (q[:, :1].expand(2, 9, 4, 64), k, v, o), (q.int(), k, v, o)):
        with pytest.raises(ValueError):
            B.checkpoint(*bad)
    with pytest.raises(B.AttnError) as e:
        B.checkpoint(q[..., :40].contiguous(), k[..., :40].contiguous(), v, o)
    assert e.value.status == B.ATTN_ERR_UNSUPPORTED_HEADDIM
    c = B.checkpoint(q, k, v, o)
    with pytest.raises(ValueError):
        B.checkpoint(q, k, v, o, out=c._replace(q_exp=c.k_exp))
    with pytest.raises(ValueError):
        B.checkpoint(q, k, v, o, out=c._replace(q=c.q.view(torch.uint8)))
    lse = torch.zeros((2, 4, 9), device="cuda")
    for args in ((c, o.float()[..., :32], lse), (c, o, lse[:, :2]), (c, o[:, :5], lse), (tuple(c)[:7], o, lse)):
        with pytest.raises((ValueError, AttributeError)):
            B.attn_backward_checkpoint(*args, scale=0.1)
    with pytest.raises(ValueError):
        B.attn_backward_checkpoint(c, o, lse, scale=0.1, cu_seqlens_q=torch.zeros(2, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ backward

def forward(xs, kw, hq, scale, dtype):
    o, lse = R.attn_forward(xs[0], xs[1], xs[2], scale, **kw)
    return o.to(dtype), lse.to(torch.float32)


def problem(dtype, b, sq, sk, hq, hkv, dqk, dv, seed, segments=None, **kw):
    """q, k, v, dO and the oracle's O and LSE on the CPU."""
    g = torch.Generator().manual_seed(seed)
    lead_q, lead_k = ((b, sq), (b, sk)) if segments is None else ((sum(segments[0]),), (sum(segments[1]),))
    sh = shapes_of(lead_q, lead_k, hq, hkv, dqk, dv)
    q, k, v, do = (torch.randn(s, generator=g).to(dtype) for s in sh)
    if segments is not None:
        cu = lambda n: torch.tensor([0] + list(n)).cumsum(0).to(torch.int32)   # noqa: E731
        kw.update(cu_seqlens_q=cu(segments[0]), cu_seqlens_k=cu(segments[1]))
    o, lse = forward((q, k, v), kw, hq, dqk ** -0.5, dtype)
    return q, k, v, o, do, lse, kw


def on_gpu(kw, segments):
    out = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in kw.items()}
    if segments is not None:
        out.update(max_seqlen_q=max(segments[0]), max_seqlen_k=max(segments[1]))
    return out


BACKWARDS = [
    # dtype, b, sq, sk, hq, hkv, dqk, dv, mask, left, right
    (torch.bfloat16, 1, 1, 1, 1, 1, 64, 64, 0, -1, -1), (torch.bfloat16, 2, 130, 130, 4, 2, 128, 128, 1, -1, -1),
    (torch.float16, 1, 257, 300, 3, 1, 64, 64, 2, -1, -1), (torch.float16, 2, 65, 200, 4, 4, 192, 128, 3, 20, 5),
    (torch.bfloat16, 1, 150, 90, 2, 1, 256, 256, 2, -1, -1),      # the first 60 rows see nothing
    (torch.float32, 2, 70, 70, 4, 2, 64, 32, 1, -1, -1), (torch.float32, 1, 33, 90, 2, 2, 32, 64, 3, 7, 0),
]


@pytest.mark.parametrize("dtype,b,sq,sk,hq,hkv,dqk,dv,mask,left,right", BACKWARDS)
@pytest.mark.parametrize("det", [1, 2])
def test_backward_is_attn_backwards_at_the_values(B, dtype, b, sq, sk, hq, hkv, dqk, dv, mask, left, right, det):
    q, k, v, o, do, lse, kw = problem(dtype, b, sq, sk, hq, hkv, dqk, dv, sq, mask=mask, left=left, right=right)
    c = B.checkpoint(*(x.cuda() for x in (q, k, v, o)))
    got = B.attn_backward_checkpoint(c, do.cuda(), lse.cuda(), scale=dqk ** -0.5, deterministic=det, **kw)
    at = [ckpt_ref.values(getattr(c, n).cpu(), getattr(c, n + "_exp").cpu(), dtype) for n in NAMES]
    for x in at:      # exact in the type
        assert torch.equal(x.to(dtype).to(F64), x)
    wide = [x.to(dtype).cuda() for x in at]
    same = B.attn_backward(*wide, do.cuda(), lse.cuda(), scale=dqk ** -0.5, deterministic=det, **kw)
    for a, x in zip(got, same):
        assert torch.equal(a, x)
    ref = R.attn_backward(*at, do, lse, dqk ** -0.5, **kw)
    tol, cos = tolerances(dtype)
    assert_all_ok([compare(g.cpu(), r, tol, cos, call_scale(ref)) for g, r in zip(got, ref)])


SEGMENTS = [([1, 0, 129, 64], [1, 5, 129, 70]), ([200, 3], [0, 300])]


@pytest.mark.parametrize("segments", SEGMENTS)
@pytest.mark.parametrize("dtype,dqk,dv", [(torch.bfloat16, 128, 128), (torch.float16, 192, 128), (torch.float32, 64, 64)])
def test_backward_of_packed_segments(B, segments, dtype, dqk, dv):
    q, k, v, o, do, lse, kw = problem(dtype, 0, 0, 0, 4, 2, dqk, dv, 5, segments=segments, mask=2)
    c = B.checkpoint(*(x.cuda() for x in (q, k, v, o)))
    gkw = on_gpu(kw, segments)
    got = B.attn_backward_checkpoint(c, do.cuda(), lse.cuda(), scale=dqk ** -0.5, deterministic=1, **gkw)
    wide = [ckpt_ref.values(getattr(c, n).cpu(), getattr(c, n + "_exp").cpu(), dtype).to(dtype).cuda() for n in NAMES]
    same = B.attn_backward(*wide, do.cuda(), lse.cuda(), scale=dqk ** -0.5, deterministic=1, **gkw)
    for a, x in zip(got, same):
        assert torch.equal(a, x)


@pytest.mark.parametrize("det", [0, 1])
def test_backward_of_padded_segments(B, det):
    """Segments with padding behind them: their rows' gradients, zeros elsewhere."""
    g = torch.Generator().manual_seed(6)
    lens, starts, rows = [50, 0, 129, 7], [0, 60, 64, 200, 230], 240
    q, k, v, do = (torch.zeros((rows, h, 64)).bfloat16() for h in (4, 2, 2, 4))
    for x in (q, k, v, do):
        for n, s in zip(lens, starts):
            x[s:s + n] = torch.randn((n, *x.shape[1:]), generator=g).bfloat16()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    pad = torch.tensor(starts, dtype=torch.int32).cuda()
    kw = dict(scale=0.125, mask=2, cu_seqlens_q=cu, cu_seqlens_k=cu, cu_seqlens_q_padded=pad, cu_seqlens_k_padded=pad,
              max_seqlen_q=129, max_seqlen_k=129)
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = B.attn_forward(*dev, **kw)
    c = B.checkpoint(*dev, o)
    wide = [ckpt_ref.values(getattr(c, n).cpu(), getattr(c, n + "_exp").cpu(), torch.bfloat16).bfloat16().cuda() for n in NAMES]
    got = B.attn_backward_checkpoint(c, do.cuda(), lse, deterministic=det, **kw)
    same = B.attn_backward(*wide, do.cuda(), lse, deterministic=1, **kw)
    for a, x in zip(got, same):
        if det:
            assert torch.equal(a, x)
        else:      # atomics: at most two fp32 partials a query tile here, so a rounding of bf16
            assert float((a.float() - x.float()).abs().max()) <= 2.0 ** -7 * float(x.float().abs().max())
    assert float(got[0][50:64].float().abs().max()) == 0 and float(got[1][207:].float().abs().max()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_backward_of_rows_that_see_one_key(B, dtype):
    """o is v, and so are their checkpoints: dQ and dK are 0 but for the order of two equal
    fp32 sums of d products, each off by at most d 2^-24 of the products' magnitudes; P is
    below 2, and a rounding of dS and of the result adds less than that again."""
    q, k, v, o, do, lse, kw = problem(dtype, 5, 1, 1, 4, 2, 128, 128, 3)
    c = B.checkpoint(*(x.cuda() for x in (q, k, v, o)))
    dq, dk, dv = (x.cpu().to(F64) for x in B.attn_backward_checkpoint(c, do.cuda(), lse.cuda(), scale=128 ** -0.5))
    wide = {n: ckpt_ref.values(getattr(c, n).cpu(), getattr(c, n + "_exp").cpu(), dtype).to(F64) for n in NAMES}
    kk, vv = (wide[n].repeat_interleave(2, 2) for n in ("k", "v"))
    assert torch.equal(wide["o"], vv)
    ds = 4 * 2 * 128 * 2.0 ** -24 * (do.to(F64) * vv).abs().sum(-1, keepdim=True) * 128 ** -0.5
    assert bool((dq.abs() <= ds * kk.abs() + 2.0 ** -24).all())
    assert bool((dk.abs() <= (ds * wide["q"].abs()).unflatten(2, (2, 2)).sum(3) + 2.0 ** -24).all())
    assert float(dv.abs().max()) > 0


@pytest.mark.parametrize("layout", ["BHSD", "SBHD"])
def test_backward_of_other_layouts(B, layout):
    q, k, v, o, do, lse, kw = problem(torch.bfloat16, 2, 100, 100, 4, 2, 64, 64, 9, mask=1)
    turn = lambda x: laid_out(x.cuda(), layout, 64)   # noqa: E731
    got = B.attn_backward_checkpoint(B.checkpoint(*map(turn, (q, k, v, o))), turn(do), lse.cuda(), scale=0.125,
                                     deterministic=1, **kw)
    plain = B.attn_backward_checkpoint(B.checkpoint(*(x.cuda() for x in (q, k, v, o))), do.cuda(), lse.cuda(), scale=0.125,
                                       deterministic=1, **kw)
    for a, x in zip(got, plain):
        assert torch.equal(a, x)
    assert got[0].stride() == turn(q).stride()


def test_backward_with_bias_and_dropout(B):
    q, k, v, o, do, lse, kw = problem(torch.bfloat16, 2, 90, 120, 4, 2, 128, 128, 11, mask=2)
    g = torch.Generator().manual_seed(1)
    bias = torch.randn((1, 4, 90, 120), generator=g).to(torch.bfloat16).cuda()
    seed, off = torch.tensor([77], device="cuda"), torch.tensor([3], device="cuda")
    extra = dict(bias=bias, dropout_p=0.2, philox_seed=seed, philox_offset=off, scale=128 ** -0.5, mask=2)
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = B.attn_forward(*dev, **extra)
    c = B.checkpoint(*dev, o)
    wide = [ckpt_ref.values(getattr(c, n).cpu(), getattr(c, n + "_exp").cpu(), torch.bfloat16).bfloat16().cuda() for n in NAMES]
    got = B.attn_backward_checkpoint(c, do.cuda(), lse, deterministic=1, return_dbias=True, **extra)
    same = B.attn_backward(*wide, do.cuda(), lse, deterministic=1, return_dbias=True, **extra)
    assert len(got) == 4
    for a, x in zip(got, same):
        assert torch.equal(a, x)


def test_backward_without_rows(B):
    z = lambda n, h: torch.zeros((2, n, h, 64), dtype=torch.bfloat16, device="cuda")   # noqa: E731
    q, k = torch.randn((2, 30, 4, 64), device="cuda").bfloat16(), torch.randn((2, 20, 2, 64), device="cuda").bfloat16()
    c = B.checkpoint(q, z(0, 2), z(0, 2), q)
    dq, dk, dv = B.attn_backward_checkpoint(c, q, torch.full((2, 4, 30), -math.inf, device="cuda"), scale=1.0)
    assert float(dq.abs().max()) == 0 and dk.numel() == 0
    c = B.checkpoint(z(0, 4), k, k, z(0, 4))
    dq, dk, dv = B.attn_backward_checkpoint(c, z(0, 4), torch.zeros((2, 4, 0), device="cuda"), scale=1.0)
    assert dq.numel() == 0 and float(dk.abs().max()) == 0 and float(dv.abs().max()) == 0


def test_status_reports_bad_segments(B):
    q, k, v, o, do, lse, kw = problem(torch.bfloat16, 0, 0, 0, 2, 2, 64, 64, 5, segments=([20, 30], [20, 30]), mask=1)
    c = B.checkpoint(*(x.cuda() for x in (q, k, v, o)))
    cu = torch.tensor([0, 20, 80], dtype=torch.int32, device="cuda")
    with pytest.raises(B.AttnError) as e:
        B.attn_backward_checkpoint(c, do.cuda(), lse.cuda(), scale=0.125, cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=30,
                                   max_seqlen_k=30, mask=1)
    assert e.value.status == B.ATTN_ERR_BAD_SEQLENS


def test_gradients_against_differences(B):
    """fp32: q, k and v that a checkpoint holds exactly, O and LSE of their forward.  The
    loss sum(dO O) is differenced in 64 bits.  What remains is O's rounding to half a
    step of its scale: it moves D_i by at most E_i = sum_c |dO_ic| step_ic / 2, hence
    dq_ic by s E_i sum_j P_ij |k_jc| and dk_jc by s sum_i E_i P_ij |q_ic|; dv not at all.  The
    fp32 kernel adds at most (terms + 16) 2^-23 of the sums of magnitudes, and the
    central difference h^2 times a third derivative: with h = 2^-12 below 1e-6 here."""
    g = torch.Generator().manual_seed(4)
    n, d, scale = 24, 32, 0.25
    q, k, v = (torch.randint(-127, 128, (1, n, 1, d), generator=g).double() / 64 for _ in range(3))
    do = torch.randn((1, n, 1, d), generator=g, dtype=F64).float().double()
    o, lse = R.attn_forward(q, k, v, scale, mask=1)
    c = B.checkpoint(*(x.float().cuda() for x in (q, k, v, o)))
    for name, x in (("q", q), ("k", k), ("v", v)):
        held = ckpt_ref.values(getattr(c, name).cpu(), getattr(c, name + "_exp").cpu(), torch.float32)
        assert torch.equal(held, x)
    got = B.attn_backward_checkpoint(c, do.float().cuda(), lse.float().cuda(), scale=scale, mask=1, deterministic=1)
    step = torch.exp2(c.o_exp.cpu().double() - 127)
    E = (do.abs().unflatten(-1, (-1, 32)) * step[..., None] / 2).sum((-1, -2))[0, :, 0]
    s = scale * q[0, :, 0] @ k[0, :, 0].T
    P = torch.exp(s - lse[0, 0][:, None]).tril()
    dP = do[0, :, 0] @ v[0, :, 0].T
    size = P * (dP.abs() + (do * o).abs().sum(-1)[0]) * scale
    K, Q = k[0, :, 0].abs(), q[0, :, 0].abs()
    noise = (n + d + 16) * 2.0 ** -23 * (1 + s.abs().max())
    bounds = (scale * E[:, None] * (P @ K) + noise * (size @ K), scale * (P * E[:, None]).T @ Q + noise * (size.T @ Q),
              noise * (P.T @ do[0, :, 0].abs()))
    h = 2.0 ** -12
    for which, (x, grad, bound) in enumerate(zip((q, k, v), got, bounds)):
        for i, col in [(0, 0), (3, 7), (11, 31), (n - 1, 5), (n // 2, 16), (1, 1)]:
            losses = []
            for sign in (1, -1):
                y = [q.clone(), k.clone(), v.clone()]
                y[which][0, i, 0, col] += sign * h
                losses.append(float((R.attn_forward(*y, scale, mask=1)[0] * do).sum()))
            want = (losses[0] - losses[1]) / (2 * h)
            assert abs(float(grad[0, i, 0, col]) - want) <= float(bound[i, col]) + 1e-6, (which, i, col)


def test_captured_and_on_another_stream(B):
    xs = [x.cuda() for x in randoms(shapes_of((2, 200), (2, 200), 4, 2, 128, 128), torch.bfloat16, 3, spread=2)]
    do = torch.randn((2, 200, 4, 128), device="cuda").bfloat16()
    kw = dict(scale=0.05, mask=1, deterministic=1, check_status=False)
    o, lse = B.attn_forward(*xs[:3], scale=0.05, mask=1)
    want = B.attn_backward_checkpoint(B.checkpoint(*xs[:3], o), do, lse, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = B.checkpoint(*xs[:3], o, stream=side)
    there = B.attn_backward_checkpoint(c, do, lse, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, there):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    held = [x.clone() for x in (*xs[:3], o, do, lse)]
    with torch.cuda.graph(graph):
        c = B.checkpoint(*held[:4])
        got = B.attn_backward_checkpoint(c, held[4], held[5], **kw)
    for x in held[:3]:
        x.mul_(0.5)
    held[3].copy_(B.attn_forward(*held[:3], scale=0.05, mask=1)[0])
    held[5].copy_(B.attn_forward(*held[:3], scale=0.05, mask=1)[1])
    for _ in range(2):
        graph.replay()
    fresh = B.attn_backward_checkpoint(B.checkpoint(*held[:4]), held[4], held[5], **kw)
    for a, b in zip(got, fresh):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(B):
    """More than 2^31 numbers in a tensor: the last rows are right."""
    rows, h, d = (1 << 31) // (32 * 128) + 3, 32, 128
    q = torch.zeros((rows, h, d), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((5, h, d), generator=torch.Generator().manual_seed(1)).bfloat16()
    q[-5:] = tail.cuda()
    small = torch.zeros((4, 1, d), dtype=torch.bfloat16, device="cuda")
    c = B.checkpoint(q, small, small, q)
    want, byte = ckpt_ref.quantise(tail)
    for n in ("q", "o"):
        assert torch.equal(getattr(c, n)[-5:].cpu(), want) and torch.equal(getattr(c, n + "_exp")[-5:].cpu(), byte)


def test_backward_in_another_type(B):
    """fp16 gradients from a checkpoint of bf16 tensors: those at the values that fp16 has,
    past 65504 limited and below 2^-24 rounded."""
    g = torch.Generator().manual_seed(8)
    q, k, v, o, do = (torch.randn((2, 70, h, 64), generator=g).bfloat16() for h in (4, 2, 2, 4, 4))
    v[0, 3, 0, 5], v[1, 60, 1, 40], k[0, 7, 1, 32:] = 1e5, -3e38, 3e-8
    lse = 4 + torch.randn((2, 4, 70), generator=g)
    c = B.checkpoint(*(x.cuda() for x in (q, k, v, o)))
    at = [ckpt_ref.values(getattr(c, n).cpu(), getattr(c, n + "_exp").cpu(), torch.float16).half() for n in NAMES]
    assert float(at[2][0, 3, 0, 5]) == 65504 and float(at[2][1, 60, 1, 40]) == -65504
    kw = dict(scale=0.125, mask=1, deterministic=1)
    small = (do.float() * 1e-4).half().cuda()
    got = B.attn_backward_checkpoint(c, small, lse.cuda(), **kw)
    same = B.attn_backward(*(x.cuda() for x in at), small, lse.cuda(), **kw)
    for a, x in zip(got, same):
        assert a.dtype == torch.float16 and bool(torch.isfinite(x).all()) and torch.equal(a, x)
