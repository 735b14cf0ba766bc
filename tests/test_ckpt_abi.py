"""8-bit checkpoints without a GPU: the structs, what the entries refuse before
anything touches the device, and the oracle's own properties."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from head_attention_backward_gb300 import binding as B
from oracle import ckpt_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x100000 * (i + 1) for i in range(24)]      # fake, aligned addresses
WS = 0x40000000
STRUCTS = {"attn_checkpoint": B.AttnCheckpointTensors, "attn_checkpoint_params": B.AttnCheckpointParams}


def test_ctypes_structs_match_c_layout():
    lines = []
    for s, c in STRUCTS.items():
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));' for f in c._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "attn_bwd.h"\nint main(void) {' + "".join(lines) + "return 0;}"
    tmp = os.path.join(ROOT, "head_attention_backward_gb300", "_build")
    os.makedirs(tmp, exist_ok=True)
    src, exe = os.path.join(tmp, "ckpt_layout.c"), os.path.join(tmp, "ckpt_layout")
    with open(src, "w") as f:
        f.write(prog)
    r = subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", src, "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0:
        pytest.skip("gcc/CUDA headers unavailable: " + r.stderr[:200])
    for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines():
        key, n = line.split()
        s, _, field = key.partition(".")
        want = getattr(STRUCTS[s], field).offset if field else ctypes.sizeof(STRUCTS[s])
        assert int(n) == want, key


def fill(p, base, kw):
    base.update(kw)
    for n, v in base.items():
        if n.startswith("stride"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    return p


def tensors(**kw):
    names = ("q", "k", "v", "o", "q_exp", "k_exp", "v_exp", "o_exp")
    return fill(B.AttnCheckpointTensors(), {n: A[i] for i, n in enumerate(names)}, kw)


def save_params(ckpt=None, **kw):
    base = dict(dtype=B.ATTN_BF16, batch=2, nhead_q=4, nhead_kv=2, seqlen_q=10, seqlen_k=12, d_qk=64, d_v=64,
                q=A[8], k=A[9], v=A[10], o=A[11])
    p = fill(B.AttnCheckpointParams(), base, kw)
    p.ckpt = tensors(**(ckpt or {}))
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(batch=0), -1), (dict(nhead_q=0), -1), (dict(nhead_kv=0), -1),
    (dict(seqlen_q=-1), -1), (dict(seqlen_k=-1), -1), (dict(batch=2 ** 20, seqlen_q=2 ** 20), -1),
    (dict(batch=1, seqlen_k=2 ** 30, nhead_kv=2 ** 10), -1),
    (dict(d_qk=0), -2), (dict(d_qk=48), -2), (dict(d_v=288), -2), (dict(d_v=-32), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(o=None), -1), (dict(q=A[8] + 8), -1),
    (dict(stride_q=(2560, 256, 60)), -1), (dict(stride_k=(2560, 0, 64)), -1), (dict(stride_v=(-2560, 128, 64)), -1),
    (dict(ckpt=dict(q=None)), -1), (dict(ckpt=dict(o_exp=None)), -1), (dict(ckpt=dict(v=A[2] + 4)), -1),
    (dict(ckpt=dict(stride_q=(5120, 256, 64))), -1),       # a gap between the batch entries
    (dict(ckpt=dict(stride_k=(1536, 128, 96))), -1),       # heads that overlap the next row
    (dict(ckpt=dict(stride_o=(0, 256, 64))), -1),
])
def test_save_refusals(lib, kw, status):
    assert B.attn_checkpoint_save(save_params(**kw)) == status


def test_save_without_rows_needs_no_tensors(lib):
    none = dict(q=None, k=None, v=None, o=None)
    assert B.attn_checkpoint_save(save_params(seqlen_q=0, seqlen_k=0, ckpt=none, **none)) == 0
    assert lib.attn_checkpoint_save(None, None) == -1


def bwd_params(**kw):
    base = dict(dtype=B.ATTN_BF16, batch=2, nhead_q=4, nhead_kv=2, seqlen_q=10, seqlen_k=12, d_qk=64, d_v=64,
                softmax_scale=0.1, dout=A[12], lse=A[13], dq=A[14], dk=A[15], dv=A[16], deterministic=1)
    return fill(B.AttnBwdParams(), base, kw)


SEGMENTS = dict(cu_seqlens_q=A[17], cu_seqlens_k=A[18], total_q=20, total_k=24)


def test_backward_workspace_is_attn_bwds_and_the_expanded_tensors(lib):
    for dtype, size, o in ((B.ATTN_BF16, 2, 0), (B.ATTN_FP16, 2, 0), (B.ATTN_FP32, 4, 1)):
        for kw in ({}, SEGMENTS):
            p = bwd_params(dtype=dtype, **kw)
            st, n = B.attn_bwd_checkpoint_workspace_size(p, tensors())
            assert st == 0
            up = lambda x: (x + 255) // 256 * 256   # noqa: E731
            q, k = 2 * 10 * 4 * 64 * size, 2 * 12 * 2 * 64 * size
            assert n == B.attn_bwd_workspace_size(p)[1] + up(q) + 2 * up(k) + o * up(q)


@pytest.mark.parametrize("kw,ckpt,status", [
    (dict(q=A[8]), {}, -1), (dict(o=A[8]), {}, -1), (dict(stride_q=(2560, 256, 64)), {}, -1),
    (dict(dtype=3), {}, -1), (dict(deterministic=3), {}, -1), (dict(softmax_scale=0.0), {}, -1),
    (dict(dout=None), {}, -1), (dict(lse=None), {}, -1), (dict(dq=A[14] + 8), {}, -1),
    (dict(d_qk=96, d_v=96), {}, -2), (dict(dtype=B.ATTN_FP32, d_qk=36), {}, -2),
    (dict(dtype=B.ATTN_FP32, d_v=128), {}, -2),
    ({}, dict(q=None), -1), ({}, dict(k_exp=None), -1), ({}, dict(o=A[3] + 8), -1),
    ({}, dict(stride_q=(5120, 256, 64)), -1),
    ({}, dict(stride_q=(2560, 64, 640)), -1),              # heads outside rows, next to contiguous tensors
    (dict(mask=4), {}, -1), (dict(dropout_p=1.0), {}, -1),
])
def test_backward_refusals(lib, kw, ckpt, status):
    p, c = bwd_params(**kw), tensors(**ckpt)
    assert B.attn_bwd_checkpoint(p, c, WS, 1 << 30) == status


def test_backward_refuses_a_bad_workspace(lib):
    p, c = bwd_params(), tensors()
    n = B.attn_bwd_checkpoint_workspace_size(p, c)[1]
    assert B.attn_bwd_checkpoint(p, c, WS, n - 1) == -3
    assert B.attn_bwd_checkpoint(p, c, 0, n) == -1
    assert B.attn_bwd_checkpoint(p, c, WS + 16, n) == -1
    assert lib.attn_bwd_checkpoint(None, ctypes.byref(c), WS, n, None) == -1
    assert lib.attn_bwd_checkpoint(ctypes.byref(p), None, WS, n, None) == -1


def test_oracle_steps_and_errors():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((50, 3, 96), generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-20, 20, (50, 3, 1), generator=g))
    x[0, 0] = 0
    x[1, 0, :32] = 127 * 2.0 ** 5
    x[2, 0, 40] = math.inf
    n, e = ckpt_ref.quantise(x)
    y = ckpt_ref.values(n, e, torch.float32)
    amax = x.unflatten(-1, (-1, 32)).abs().amax(-1)
    step = torch.exp2(e.double() - 127)
    fine = e != 255
    assert bool((n.unflatten(-1, (-1, 32)).abs().amax(-1) <= 127).all())
    # least scales: the one below would not hold the largest magnitude
    assert bool((amax[fine] <= 127 * step[fine]).all()) and bool(((amax > 63.5 * step) | (e == 1))[fine].all())
    err = (x - y).unflatten(-1, (-1, 32)).abs().amax(-1)
    assert bool((err[fine] <= step[fine] / 2).all())
    assert int((~fine).sum()) == 1 and bool(torch.isnan(y[2, 0, 32:64]).all()) and not bool(torch.isnan(y[2, 0, :32]).any())
    # what is read back is stored again without a change
    n2, e2 = ckpt_ref.quantise(torch.where(torch.isnan(y), torch.zeros_like(y), y))
    assert bool((ckpt_ref.values(n2, e2, torch.float32)[..., :32] == y[..., :32])[3:].all())
