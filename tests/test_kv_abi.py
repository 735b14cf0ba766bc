"""What the serving operators refuse, and their structs, without a GPU: every
check runs before anything touches the device."""
import ctypes
import os
import subprocess

import pytest
import torch

from head_attention_backward_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"attn_rope_params": B.AttnRopeParams, "attn_kv_cache": B.AttnKvCache,
           "attn_kv_plan_params": B.AttnKvPlanParams, "attn_kv_append_params": B.AttnKvAppendParams,
           "attn_kv_fwd_params": B.AttnKvFwdParams}


def test_ctypes_structs_match_c_layout():
    lines = []
    for s, c in STRUCTS.items():
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));' for f in c._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "attn_bwd.h"\nint main(void) {' + "".join(lines) + "return 0;}"
    tmp = os.path.join(ROOT, "head_attention_backward_gb300", "_build")
    os.makedirs(tmp, exist_ok=True)
    src, exe = os.path.join(tmp, "kv_layout.c"), os.path.join(tmp, "kv_layout")
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


# fake, aligned addresses: the checks never dereference device pointers
A = [0x100000 * (i + 1) for i in range(12)]
FREQ = (ctypes.c_double * 128)(*([0.5] * 128))
AXIS = (ctypes.c_uint8 * 128)(*([1] * 128))


def rope_params(**kw):
    base = dict(dtype=B.ATTN_BF16, batch=1, seqlen=10, nhead_q=4, nhead_kv=2, head_dim=64, rot_dim=64, n_axes=2,
                positions=A[0], inv_freq=ctypes.addressof(FREQ), pair_axis=ctypes.addressof(AXIS), q=A[1], k=A[2],
                q_out=A[3], k_out=A[4])
    base.update(kw)
    p = B.AttnRopeParams()
    for n, v in base.items():
        if n.startswith("stride"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    return p


BAD_FREQ = (ctypes.c_double * 128)(*([float("nan")] * 128))


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(batch=-1), -1), (dict(seqlen=-1), -1), (dict(nhead_q=0), -1),
    (dict(nhead_kv=-1), -1), (dict(batch=2 ** 20, seqlen=2 ** 20), -1),
    (dict(head_dim=0), -2), (dict(head_dim=257), -2), (dict(head_dim=264), -2), (dict(head_dim=60, rot_dim=20), -2),
    (dict(rot_dim=0), -1), (dict(rot_dim=63), -1), (dict(rot_dim=66), -1), (dict(n_axes=0), -1), (dict(n_axes=5), -1),
    (dict(n_axes=1), -1), (dict(inv_freq=None), -1), (dict(inv_freq=ctypes.addressof(BAD_FREQ)), -1),
    (dict(positions=None), -1), (dict(positions=A[0] + 2), -1), (dict(stride_pos=(-1, 0, 0)), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(q_out=None), -1), (dict(k_out=None), -1), (dict(q=A[1] + 2), -1),
    (dict(stride_q=(640, 60, 64)), -1), (dict(stride_q=(640, 0, 64)), -1), (dict(stride_k_out=(0, -64, 64)), -1),
    (dict(q_out=A[1], stride_q_out=(0, 512, 64)), -1),
])
def test_rope_refusals(lib, kw, status):
    assert B.attn_rope(rope_params(**kw)) == status


def test_rope_without_rows_needs_no_tensors(lib):
    assert B.attn_rope(rope_params(seqlen=0, q=None, k=None, q_out=None, k_out=None, positions=None)) == 0
    assert lib.attn_rope(None, None) == -1


def cache(**kw):
    base = dict(num_pages=10, page_size=16, nhead_kv=2, d_qk=128, d_v=128, k=A[5], v=A[6], k_exp=A[7], v_exp=A[8])
    base.update(kw)
    c = B.AttnKvCache()
    for n, v in base.items():
        if n.startswith("stride"):
            getattr(c, n)[:] = v
        else:
            setattr(c, n, v)
    return c


BAD_CACHES = [
    (dict(num_pages=0), -1), (dict(nhead_kv=0), -1), (dict(nhead_kv=16385), -1),
    (dict(page_size=8), -1), (dict(page_size=48), -1),
    (dict(page_size=512), -1), (dict(d_qk=96), -2), (dict(d_qk=64), -2), (dict(d_v=64), -2), (dict(reserved=1), -1),
]
BAD_CACHE_POINTERS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_exp=None), -1), (dict(v_exp=None), -1), (dict(k=A[5] + 8), -1),
    (dict(v=A[6] + 1), -1), (dict(stride_k=(4096, 256, 0)), -1), (dict(stride_k=(4096, 256, 120)), -1),
    (dict(stride_v=(-4096, 256, 128)), -1),
]


def plan_params(**kw):
    base = dict(batch=3, page_size=16, num_pages=10, max_blocks=4, max_tokens=8, table_stride=4, new_lens=A[0],
                seqlens=A[1], seqlens_out=A[1], block_table=A[2], free_pages=A[3], free_count=A[4],
                free_count_out=A[4], cu_seqlens=A[5], positions=A[6], slots=A[7], status=A[8])
    base.update(kw)
    p = B.AttnKvPlanParams()
    for n, v in base.items():
        setattr(p, n, v)
    return p


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=8193), dict(page_size=24), dict(num_pages=0), dict(max_blocks=0), dict(max_tokens=-1),
    dict(max_tokens=2 ** 30 + 1),
    dict(max_blocks=2 ** 27, table_stride=2 ** 27), dict(table_stride=3), dict(reserved=7), dict(new_lens=None),
    dict(seqlens=None), dict(seqlens_out=None), dict(block_table=None), dict(free_pages=None), dict(free_count=None),
    dict(free_count_out=None), dict(cu_seqlens=None), dict(positions=None), dict(slots=None), dict(status=None),
    dict(slots=A[7] + 4), dict(seqlens=A[1] + 1)])
def test_plan_refusals(lib, kw):
    assert B.attn_kv_plan(plan_params(**kw)) == -1
    assert lib.attn_kv_plan(None, None) == -1


def append_params(cache_kw=None, **kw):
    base = dict(dtype=B.ATTN_FP16, tokens=4, k=A[0], v=A[1], slots=A[2])
    base.update(kw)
    p = B.AttnKvAppendParams()
    for n, v in base.items():
        if n.startswith("stride"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    p.cache = cache(**(cache_kw or {}))
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=B.ATTN_FP32), -1), (dict(dtype=9), -1), (dict(tokens=-1), -1), (dict(tokens=2 ** 30 + 1), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(slots=A[2] + 4), -1), (dict(k=A[0] + 8), -1),
    (dict(stride_k=(0, 250, 128)), -1), (dict(stride_v=(0, 256, 0)), -1)]
    + [(dict(cache_kw=c), s) for c, s in BAD_CACHES + BAD_CACHE_POINTERS])
def test_append_refusals(lib, kw, status):
    assert B.attn_kv_append(append_params(**kw)) == status


def test_append_without_tokens(lib):
    assert B.attn_kv_append(append_params(tokens=0, k=None, v=None, slots=None)) == 0
    assert lib.attn_kv_append(None, None) == -1


def fwd_params(cache_kw=None, **kw):
    base = dict(dtype=B.ATTN_BF16, batch=3, nhead_q=8, total_q=3, max_seqlen_q=1, max_seqlen_k=100, max_blocks=7,
                mask=2, window_left=-1, window_right=-1, softmax_scale=0.1, cu_seqlens_q=A[0], seqlens_k=A[1],
                block_table=A[2], table_stride=7, q=A[3], o=A[4], lse=A[9])
    base.update(kw)
    p = B.AttnKvFwdParams()
    for n, v in base.items():
        if n.startswith("stride"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    p.cache = cache(**(cache_kw or {}))
    return p


SIZES = [
    (dict(dtype=B.ATTN_FP32), -1), (dict(batch=0), -1), (dict(batch=2 ** 20 + 1), -1), (dict(nhead_q=0), -1),
    (dict(nhead_q=7), -1), (dict(total_q=-1), -1), (dict(max_seqlen_q=-1), -1), (dict(max_seqlen_k=-1), -1),
    (dict(max_blocks=0), -1), (dict(max_blocks=2 ** 27, table_stride=2 ** 27), -1), (dict(mask=4), -1),
    (dict(mask=-1), -1), (dict(mask=3, window_left=-2), -1), (dict(mask=3, window_right=-2), -1),
    (dict(softmax_scale=0.0), -1), (dict(softmax_scale=float("inf")), -1), (dict(softmax_scale=float("nan")), -1),
    (dict(reserved=1), -1), (dict(max_seqlen_q=2 ** 30, total_q=2 ** 30), -1)]


@pytest.mark.parametrize("kw,status", SIZES + [(dict(cache_kw=c), s) for c, s in BAD_CACHES])
def test_fwd_sizes_refused(lib, kw, status):
    p = fwd_params(**kw)
    assert B.attn_kv_fwd_workspace_size(p) == (status, 0)
    assert B.attn_kv_fwd(p, A[10], 1 << 40) == status
    assert B.attn_kv_fwd_read_status(p, A[10], 1 << 40)[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(cu_seqlens_q=None), -1), (dict(seqlens_k=None), -1), (dict(block_table=None), -1), (dict(table_stride=6), -1),
    (dict(q=None), -1), (dict(o=None), -1), (dict(lse=None), -1), (dict(q=A[3] + 8), -1), (dict(o=A[4] + 2), -1),
    (dict(lse=A[9] + 2), -1), (dict(cu_seqlens_q=A[0] + 1), -1), (dict(cu_seqlens_q_padded=A[0] + 2), -1),
    (dict(stride_q=(0, 1004, 128)), -1), (dict(stride_o=(0, 1024, 4)), -1)]
    + [(dict(cache_kw=c), s) for c, s in BAD_CACHE_POINTERS])
def test_fwd_refusals(lib, kw, status):
    assert B.attn_kv_fwd(fwd_params(**kw), A[10], 1 << 40) == status


def test_fwd_workspace(lib):
    p = fwd_params()
    st, n = B.attn_kv_fwd_workspace_size(p)
    assert st == 0 and n >= 256
    assert B.attn_kv_fwd(p, A[10], n - 1) == B.ATTN_ERR_WORKSPACE_TOO_SMALL
    assert B.attn_kv_fwd(p, A[10] + 128, n) == -1
    assert B.attn_kv_fwd(p, 0, n) == -1
    assert B.attn_kv_fwd_read_status(p, A[10], n - 1)[0] == B.ATTN_ERR_WORKSPACE_TOO_SMALL
    assert B.attn_kv_fwd_read_status(p, 0, n)[0] == -1
    assert lib.attn_kv_fwd_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == -1
    # a longer bound needs more splits, never less memory
    sizes = [B.attn_kv_fwd_workspace_size(fwd_params(max_seqlen_k=k, max_blocks=2 ** 16, table_stride=2 ** 16))[1]
             for k in (0, 16, 1000, 2 ** 17, 2 ** 20)]
    assert sizes == sorted(sizes)


def test_new_status_codes_have_names(lib):
    for code in (B.ATTN_ERR_BAD_PAGE, B.ATTN_ERR_OUT_OF_PAGES):
        assert B.attn_status_string(code) != "unknown status"


@pytest.fixture(scope="module")
def marshal(lib):
    from head_attention_backward_gb300 import build
    build.build_marshal()
    return B._load_marshal()


def test_marshalling_refuses_before_it_calls(marshal):
    """Wrong types, shapes, layouts and devices are Python errors; no argument
    ends the process."""
    q = torch.zeros((4, 2, 64))
    f = B.rope_frequencies(64)
    for args in ((), (1,), (None,) * 9, (q,) * 9, (q, None, q, f, None, 0, 0, None, None), ("x",) * 9):
        with pytest.raises((TypeError, ValueError)):
            marshal.rope(*args)
    for fn, n in ((marshal.cache, 4), (marshal.plan, 8), (marshal.append, 5), (marshal.attend, 17), (marshal.bind, 6)):
        for x in (None, 3.5, "x", q, torch.zeros(0), torch.zeros((), dtype=torch.int32)):
            with pytest.raises((TypeError, ValueError)):
                fn(*(x,) * n)
        with pytest.raises(TypeError):
            fn()
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.kv_plan(i, i, torch.zeros((3, 2), dtype=torch.int32), i, i[:1], page_size=16, max_tokens=4)
    with pytest.raises(ValueError):
        B.rope(q, None, torch.zeros(4, dtype=torch.int32), f)      # not on a GPU
    with pytest.raises(ValueError):
        B.KvCache(torch.zeros((2, 16, 1, 64)), torch.zeros((2, 16, 1, 64)), torch.zeros((2, 1)), torch.zeros((2, 1)))
    with pytest.raises(ValueError):
        B.KvCache(*(torch.zeros((2, 16, 1, 64), dtype=torch.uint8) for _ in range(2)),
                  *(torch.zeros((2, 1), dtype=torch.uint8) for _ in range(2)))
