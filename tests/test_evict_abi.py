"""Attention weights and eviction without a GPU: the structs, and what the
entries refuse before anything touches the device."""
import ctypes
import os
import subprocess

import pytest
import torch

from head_attention_backward_gb300 import binding as B
from oracle import evict_ref
from tests.test_kv_abi import A, BAD_CACHE_POINTERS, BAD_CACHES, ROOT, cache, plan_params

STRUCTS = {"attn_kv_weights": B.AttnKvWeights, "attn_kv_weigh_params": B.AttnKvWeighParams,
           "attn_kv_evict_params": B.AttnKvEvictParams}
WS = 0x40000000


def test_ctypes_structs_match_c_layout():
    lines = []
    for s, c in STRUCTS.items():
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));' for f in c._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "attn_bwd.h"\nint main(void) {' + "".join(lines) + "return 0;}"
    tmp = os.path.join(ROOT, "head_attention_backward_gb300", "_build")
    os.makedirs(tmp, exist_ok=True)
    src, exe = os.path.join(tmp, "evict_layout.c"), os.path.join(tmp, "evict_layout")
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


def weights(**kw):
    w = B.AttnKvWeights()
    for n, v in {**dict(weight=A[9], position=A[10], status=A[11]), **kw}.items():
        setattr(w, n, v)
    return w


def fill(p, base, kw, cache_kw, weights_kw):
    base.update(kw)
    for n, v in base.items():
        if n.startswith("stride"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    p.cache, p.weights = cache(**(cache_kw or {})), weights(**(weights_kw or {}))
    return p


def weigh_params(cache_kw=None, weights_kw=None, **kw):
    base = dict(dtype=B.ATTN_BF16, batch=3, nhead_q=8, total_q=3, max_seqlen_q=1, max_seqlen_k=100, max_blocks=7,
                mask=2, window_left=-1, window_right=-1, softmax_scale=0.1, decay=1.0, cu_seqlens_q=A[0], seqlens_k=A[1],
                block_table=A[2], table_stride=7, q=A[3], lse=A[4])
    return fill(B.AttnKvWeighParams(), base, kw, cache_kw, weights_kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=B.ATTN_FP32), -1), (dict(dtype=-1), -1), (dict(batch=0), -1), (dict(nhead_q=0), -1), (dict(nhead_q=7), -1),
    (dict(total_q=-1), -1), (dict(max_seqlen_q=-1), -1), (dict(max_seqlen_k=-1), -1), (dict(max_blocks=0), -1),
    (dict(max_blocks=2 ** 27, table_stride=2 ** 27), -1), (dict(table_stride=6), -1), (dict(mask=4), -1),
    (dict(mask=3, window_left=-2), -1), (dict(softmax_scale=0.0), -1), (dict(softmax_scale=float("nan")), -1),
    (dict(decay=-0.5), -1), (dict(decay=float("inf")), -1), (dict(decay=float("nan")), -1), (dict(batch=2 ** 24), -1),
    (dict(cu_seqlens_q=None), -1), (dict(seqlens_k=None), -1), (dict(block_table=None), -1), (dict(q=None), -1),
    (dict(lse=None), -1), (dict(q=A[3] + 8), -1), (dict(lse=A[4] + 2), -1), (dict(position_offsets=A[8] + 1), -1),
    (dict(cu_seqlens_q_padded=A[0] + 2), -1), (dict(new_lens=A[8] + 2), -1), (dict(stride_q=(0, 1004, 128)), -1),
    (dict(weights_kw=dict(weight=None)), -1), (dict(weights_kw=dict(position=None)), -1),
    (dict(weights_kw=dict(status=None)), -1), (dict(weights_kw=dict(weight=A[9] + 2)), -1)]
    + [(dict(cache_kw=c), s) for c, s in BAD_CACHES + BAD_CACHE_POINTERS])
def test_weigh_refusals(lib, kw, status):
    assert B.attn_kv_weigh(weigh_params(**kw)) == status


def test_weigh_without_tokens(lib):
    assert B.attn_kv_weigh(weigh_params(total_q=0, q=None, lse=None)) == 0
    assert lib.attn_kv_weigh(None, None) == -1


def evict_params(cache_kw=None, weights_kw=None, **kw):
    base = dict(batch=3, max_seqlen_k=100, max_blocks=7, table_stride=7, keep=A[0], seqlens=A[1], seqlens_out=A[1],
                position_offsets=A[2], position_offsets_out=A[2], block_table=A[3], free_pages=A[4], free_count=A[5],
                free_count_out=A[5], status=A[6])
    return fill(B.AttnKvEvictParams(), base, kw, cache_kw, weights_kw)


SIZES = [dict(batch=0), dict(batch=8193), dict(max_seqlen_k=-1), dict(max_blocks=0), dict(table_stride=6), dict(sink=-1),
         dict(recent=-1), dict(slack=-1), dict(reserved=1), dict(max_blocks=2 ** 27, table_stride=2 ** 27),
         dict(batch=8192, cache_kw=dict(nhead_kv=4096)), dict(cache_kw=dict(page_size=24)), dict(cache_kw=dict(num_pages=0))]


@pytest.mark.parametrize("kw", SIZES)
def test_evict_sizes_refused(lib, kw):
    assert B.attn_kv_evict_workspace_size(evict_params(**kw)) == (-1, 0)
    assert B.attn_kv_evict(evict_params(**kw), WS, 1 << 40) == -1


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), -1) for n in (
    "keep", "seqlens", "seqlens_out", "position_offsets", "position_offsets_out", "block_table", "free_pages", "free_count",
    "free_count_out", "status")] + [(dict(keep=A[0] + 1), -1), (dict(weights_kw=dict(weight=None)), -1),
                                    (dict(weights_kw=dict(position=A[10] + 2)), -1)]
    + [(dict(cache_kw=c), s) for c, s in BAD_CACHES + BAD_CACHE_POINTERS])
def test_evict_refusals(lib, kw, status):
    assert B.attn_kv_evict(evict_params(**kw), WS, 1 << 40) == status


def test_evict_workspace(lib):
    p = evict_params()
    st, n = B.attn_kv_evict_workspace_size(p)
    assert st == 0 and n >= 256
    assert B.attn_kv_evict(p, WS, n - 1) == B.ATTN_ERR_WORKSPACE_TOO_SMALL
    assert B.attn_kv_evict(p, WS + 128, n) == -1
    assert B.attn_kv_evict(p, 0, n) == -1
    assert lib.attn_kv_evict(None, WS, n, None) == -1
    assert lib.attn_kv_evict_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == -1
    wide = dict(max_blocks=2 ** 16, table_stride=2 ** 16)
    sizes = [B.attn_kv_evict_workspace_size(evict_params(max_seqlen_k=k, **wide))[1] for k in (0, 16, 1000, 2 ** 17, 2 ** 20)]
    assert sizes == sorted(sizes)


def test_plan_refuses_misaligned_offsets(lib):
    assert B.attn_kv_plan(plan_params(position_offsets=A[9] + 2)) == -1


def test_marshalling_refuses_before_it_calls(lib):
    from head_attention_backward_gb300 import build
    build.build_marshal()
    m = B._load_marshal()
    q = torch.zeros((4, 2, 64))
    for fn, n in ((m.weigh, 18), (m.evict, 15), (m.checkpoint, 5), (m.backward, 25), (m.plan, 9)):
        for x in (None, 3.5, "x", q, torch.zeros(0), torch.zeros((), dtype=torch.int32), (1, 2, 3), (q,) * 8):
            with pytest.raises((TypeError, ValueError)):
                fn(*(x,) * n)
        with pytest.raises(TypeError):
            fn()


def test_oracle_choice():
    w = torch.tensor([3.0, float("nan"), 3.0, 0.0, 9.0, -0.0, float("-inf"), 1.0])
    pos = [5, 0, 1, 2, 3, 4, 6, 7]
    assert evict_ref.stays(w, pos, 3, 0, 100) == [0, 2, 4]
    assert evict_ref.stays(w, pos, 2, 0, 100) == [0, 4]                 # of equals the lower row
    assert evict_ref.stays(w, pos, 3, 2, 7) == [1, 2, 7]                # protected first
    assert evict_ref.stays(w, pos, 2, 2, 7) == [2, 7]                   # and among themselves by weight
    assert evict_ref.stays(w, pos, 7, 0, 100) == [0, 2, 3, 4, 5, 6, 7]  # NaN below every number
