"""Inputs and tolerances shared by the tests of rotary positions and the paged
cache (no arithmetic of the operators)."""
import math

import torch

F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def random_cache(pages, page, heads, d, g, spread=3):
    """Cache half on the CPU: bytes of a normal distribution (no NaN) and
    exponents that differ from page to page and head to head."""
    x = (torch.randn((pages, page, heads, d), generator=g) * 110).clamp(-448, 448)
    e = torch.randint(127 - 8, 127 - 8 + spread, (pages, heads), generator=g).to(torch.uint8)
    return x.to(torch.float8_e4m3fn).view(torch.uint8), e


def block_table(lens, page, g, extra_pages=2, extra_cols=1):
    need = [(n + page - 1) // page for n in lens]
    order = torch.randperm(sum(need) + extra_pages, generator=g).tolist()
    cols = max(max(need), 1) + extra_cols
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (cols - n))
        at += n
    return table, sum(need) + extra_pages


def attend_bounds(o, lse, mag, size, dtype, d_qk, keys, weight_type):
    """Largest deviations of O and LSE, element by element.

    A score is a d_qk-term sum of exact products in fp32 accumulators: its
    error is at most d_qk 2^-23 sum |q k| scale =: ds (truncating adds).  Each
    weight then carries a relative error of ds, of the exponent's argument (its
    magnitude, below 2^7 where the weight counts, at 2^-24, times ln 2: 2^-17),
    of ex2.approx (2^-22) and of its rounding to `weight_type` (half a step);
    O = sum p v / l moves by that times sum p |v| / l, doubled for the
    denominator's share of ds; fp32 sums of up to `keys` terms add keys / 16
    2^-24 (16 lanes and warps share them) and O's own rounding half a step."""
    ds = d_qk * 2.0 ** -23 * size                                    # [Hq, T]
    rel = 2 * ds + half_step(weight_type) + 2.0 ** -16 + (keys / 16 + 16) * 2.0 ** -24
    tol_o = rel.T[..., None] * mag + half_step(dtype) * o.abs() + 1e-30
    if dtype == torch.float16:
        tol_o = tol_o + 2.0 ** -25                                   # half a step of subnormals
    tol_l = ds + 2.0 ** -16 + (keys / 16 + 16) * 2.0 ** -24 + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)
    return tol_o, tol_l


def check_attend(got_o, got_lse, ref, dtype, d_qk, keys, weight_type=torch.float16, what=""):
    o, lse, mag, size = ref
    tol_o, tol_l = attend_bounds(o, lse, mag, size, dtype, d_qk, keys, weight_type)
    live = ~torch.isnan(lse)
    got_o, got_lse = got_o.cpu().to(F64), got_lse.cpu().to(F64)
    rows = live.T
    empty = live & (lse == -math.inf)
    assert bool((got_lse[empty] == -math.inf).all()), f"{what}: LSE of rows without keys"
    some = live & ~empty
    e = ((got_lse - lse).abs() - tol_l)[some]
    assert e.numel() == 0 or float(e.max()) <= 0, f"{what}: LSE off by {float((got_lse - lse).abs()[some].max())}"
    d = (got_o - o).abs()
    bad = (d > tol_o) & rows[..., None]
    assert not bool(bad.any()) and not bool(torch.isnan(got_o[rows]).any()), (
        f"{what}: O off by {float(d[rows].max())}, {int(bad.sum())} of {bad.numel()} beyond their bounds")
