"""Plain fp64 CPU oracle of the 8-bit activation checkpoint.

TEST INFRASTRUCTURE ONLY, like attn_ref: nothing on the product path imports
it, and it shares no code with the CUDA path.  A group is 32 consecutive
columns of a row and head; its scale 2^e is the least power of two, e >= -126,
with 127 * 2^e >= the group's largest magnitude, found by trying; its numbers
are the values over the scale, rounded half to even.  A group with an infinity
or a NaN has byte 255 and zeros.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
GROUP = 32


def quantise(x):
    """(numbers int8, exponent bytes uint8) of x [..., d]."""
    y = x.to(F64).unflatten(-1, (-1, GROUP))
    flat = y.reshape(-1, GROUP)
    numbers = torch.zeros(flat.shape, dtype=torch.int8)
    byte = torch.zeros(flat.shape[0], dtype=torch.uint8)
    top = flat.abs().amax(-1)
    for i, amax in enumerate(top.tolist()):
        if not math.isfinite(amax):
            byte[i] = 255
            continue
        e = -126
        while amax > 127 * math.ldexp(1.0, e):
            e += max(1, int(math.log2(amax / (127 * math.ldexp(1.0, e)))) - 1)
        while e > -126 and amax <= 127 * math.ldexp(1.0, e - 1):
            e -= 1
        byte[i] = e + 127
    fine = byte != 255
    step = torch.exp2(byte[fine].to(F64) - 127)[:, None]
    numbers[fine] = torch.round(flat[fine] / step).to(torch.int8)
    return numbers.view(x.shape), byte.view(*x.shape[:-1], -1)


def values(numbers, byte, dtype):
    """What they stand for, in 64 bits, limited to dtype's largest finite value."""
    step = torch.exp2(byte.to(F64) - 127)
    step = torch.where(byte == 255, torch.full_like(step, math.nan), step)
    y = numbers.to(F64).unflatten(-1, (-1, GROUP)) * step[..., None]
    top = torch.finfo(dtype).max
    return y.flatten(-2).clamp(-top, top)
