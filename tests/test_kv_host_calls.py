"""The serving entries' launches, without a GPU: their host code runs against a
stand-in for the CUDA runtime that counts launches, refuses those whose dynamic
shared memory is past the limit in force, and fails one on request."""
import ctypes
import os
import subprocess

import pytest

from head_attention_backward_gb300 import binding as B
from head_attention_backward_gb300 import build as _build
from tests.test_kv_abi import A, append_params, fwd_params, plan_params, rope_params

FAKE = r"""
#include <cuda_runtime_api.h>
#include <map>
#include <string>
#include <vector>

namespace {
struct Launch { std::string name; size_t smem; bool ok; };
std::map<const void*, std::string> names;
std::map<const void*, int> limits;               // dynamic shared memory that a kernel was allowed
std::vector<Launch> launches;
int fail_at = -1;
cudaError_t pending = cudaSuccess;
dim3 cfg_grid, cfg_block;
size_t cfg_smem;
cudaStream_t cfg_stream;

// 48 KB by default, less the kernel's static shared memory (1 KB stands for it)
cudaError_t launch(const void* f, size_t smem) {
  const int index = (int)launches.size();
  const auto l = limits.find(f);
  const size_t limit = l == limits.end() ? 47 * 1024 : l->second;
  const bool ok = index != fail_at && smem <= limit;
  launches.push_back({names[f], smem, ok});
  if (!ok) pending = cudaErrorInvalidValue;
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}
int encode(void) { return 0; }                   // a tensor map, as far as the host goes
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*) {
  names[host] = name;
}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t smem, struct CUstream_st* s) {
  cfg_grid = g, cfg_block = b, cfg_smem = smem, cfg_stream = s;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* smem, void* s) {
  *g = cfg_grid, *b = cfg_block, *smem = cfg_smem, *static_cast<cudaStream_t*>(s) = cfg_stream;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void**, size_t smem, cudaStream_t) { return launch(k, smem); }
cudaError_t cudaLaunchKernel(const void* f, dim3, dim3, void**, size_t smem, cudaStream_t) { return launch(f, smem); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) { return launch(f, c->dynamicSmemBytes); }
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) limits[f] = v;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) {
  const cudaError_t e = pending;
  pending = cudaSuccess;
  return e;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             enum cudaDriverEntryPointQueryResult* r) {
  *f = reinterpret_cast<void*>(&encode);
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void*, const void*, size_t, enum cudaMemcpyKind) { return cudaErrorNotSupported; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaErrorNotSupported; }

void fake_reset(int fail) { launches.clear(); limits.clear(); fail_at = fail; pending = cudaSuccess; }
int fake_count(void) { return (int)launches.size(); }
int fake_done(void) { int n = 0; for (const Launch& l : launches) n += l.ok; return n; }
const char* fake_name(int i) { return launches[i].name.c_str(); }
int fake_limit(const char* part) {               // of the kernel whose name contains `part`; 0: never set
  for (const auto& l : limits)
    if (names[l.first].find(part) != std::string::npos) return l.second;
  return 0;
}
}
"""

UNITS = ("kv_plan", "kv_append", "kv_fwd", "kv_long", "fwd_tc", "rope")


@pytest.fixture(scope="module")
def fake(lib, tmp_path_factory):
    """The serving entries' objects, linked with the stand-in."""
    objs = [os.path.join(_build.OUT_DIR, u + ".o") for u in UNITS]
    if not all(os.path.exists(o) for o in objs):
        _build.build_library(force=True)
    d = tmp_path_factory.mktemp("fake")
    src, so = str(d / "fake.cpp"), str(d / "libfake.so")
    with open(src, "w") as f:
        f.write(FAKE)
    inc = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic,-z,defs", "-I", inc, src, *objs, "-o", so],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    x = ctypes.CDLL(so)
    x.fake_name.restype = ctypes.c_char_p
    for n in ("attn_rope", "attn_kv_plan", "attn_kv_append", "attn_kv_fwd"):
        getattr(x, n).argtypes = getattr(lib, n).argtypes
    return x


def plan(fake, batch, max_tokens=8):
    return fake.attn_kv_plan(ctypes.byref(plan_params(batch=batch, max_tokens=max_tokens)), None)


@pytest.mark.parametrize("batch", [1, 256, 2047, 3000, 3047, 3048, 3060, 3071, 3073, 8191, 8192])
def test_plan_is_launched_at_every_batch(fake, batch):
    """As the first call of a process: whatever shared memory it needs has to be
    asked for."""
    fake.fake_reset(-1)
    assert plan(fake, batch) == 0
    assert fake.fake_done() == 1


def test_a_plan_never_lowers_the_limit_of_another(fake):
    """The limit belongs to the kernel, not to a call: a call of fewer requests on
    another thread may come between a call's setting it and its launch."""
    fake.fake_reset(-1)
    assert plan(fake, 8192) == 0
    high = fake.fake_limit(b"plan_kernel")
    assert high >= (4 * 8192 + 3) * 4
    for batch in (3073, 3100, 5000, 8192):
        assert plan(fake, batch) == 0
        assert fake.fake_limit(b"plan_kernel") == high


DECODE = dict(cache_kw=dict(num_pages=10000), max_blocks=8192, table_stride=8192)
CALLS = {
    # call, its kernels in order
    "rope": (lambda: ("attn_rope", rope_params()), ["rope_kernel"]),
    "plan, few tokens": (lambda: ("attn_kv_plan", plan_params()), ["plan_kernel"]),
    "plan, many tokens": (lambda: ("attn_kv_plan", plan_params(max_tokens=5000)), ["plan_kernel", "fill_kernel"]),
    "plan, many requests": (lambda: ("attn_kv_plan", plan_params(batch=8192, max_tokens=5000)), ["plan_kernel", "fill_kernel"]),
    "append": (lambda: ("attn_kv_append", append_params()), ["append_kernel"]),
    "attend, one split": (lambda: ("attn_kv_fwd", fwd_params()), ["kv_fwd_kernel"]),
    "attend, a cluster": (lambda: ("attn_kv_fwd", fwd_params(max_seqlen_k=1000, **DECODE)), ["kv_fwd_kernel"]),
    "attend, few rows": (lambda: ("attn_kv_fwd", fwd_params(max_seqlen_k=131072, **DECODE)), ["kv_fwd_kernel", "join_kernel"]),
    "attend, many rows": (lambda: ("attn_kv_fwd", fwd_params(batch=400, total_q=400, max_seqlen_k=131072, **DECODE)),
                          ["kv_fwd_kernel", "join_rows_kernel"]),
    "attend, a prompt": (lambda: ("attn_kv_fwd", fwd_params(batch=2, total_q=700, max_seqlen_q=600, max_seqlen_k=640, max_blocks=40,
                                                            table_stride=40)),
                         ["setup_kernel", "expand_kernel", "fwd_tc_kernel", "kv_fwd_kernel"]),
    "attend, a short prompt over many keys": (
        lambda: ("attn_kv_fwd", fwd_params(batch=1, nhead_q=2, total_q=130, max_seqlen_q=130, max_seqlen_k=5000, **DECODE)),
        ["setup_kernel", "expand_kernel", "fwd_tc_kernel", "join_parts_kernel", "kv_fwd_kernel", "join_kernel"]),
    "attend, prompts in groups": (
        lambda: ("attn_kv_fwd", fwd_params(cache_kw=dict(num_pages=10000, nhead_kv=8), batch=2, total_q=2000, max_seqlen_q=1000,
                                           max_seqlen_k=2 ** 18, max_blocks=2 ** 14, table_stride=2 ** 14)),
        ["setup_kernel"] + 2 * ["expand_kernel", "fwd_tc_kernel", "join_parts_kernel"] + ["kv_fwd_kernel"]),
}


@pytest.mark.parametrize("what", CALLS)
def test_no_kernel_follows_one_that_was_not_launched(fake, what):
    """The kernels of a call read what those before them wrote: where a launch
    fails, the call ends there with its error."""
    make, kernels = CALLS[what]

    def run(fail):
        fake.fake_reset(fail)
        name, p = make()
        more = (A[10], 1 << 40, None) if name == "attn_kv_fwd" else (None,)
        st = getattr(fake, name)(ctypes.byref(p), *more)
        return st, [fake.fake_name(i).decode() for i in range(fake.fake_count())]

    st, names = run(-1)
    assert st == 0 and len(names) == len(kernels) and all(k in n for k, n in zip(kernels, names)), names
    for i in range(len(kernels)):
        st, ran = run(i)
        assert st == B.ATTN_ERR_CUDA and ran == names[:i + 1], (i, ran)
        assert fake.fake_done() == i


@pytest.mark.parametrize("what", CALLS)
def test_a_failed_launch_is_not_held_against_the_next_call(fake, what):
    """The runtime remembers an error until it is asked for: a call that failed
    leaves none behind."""
    make, kernels = CALLS[what]
    for i in range(len(kernels)):
        fake.fake_reset(i)
        name, p = make()
        more = (A[10], 1 << 40, None) if name == "attn_kv_fwd" else (None,)
        assert getattr(fake, name)(ctypes.byref(p), *more) == B.ATTN_ERR_CUDA
        assert fake.cudaGetLastError() == 0, i


@pytest.mark.parametrize("batch,seqlen,heads", [(1, 10, 4), (3, 1, 4), (2, 5, 1), (1, 1, 1)])
def test_rope_in_place_whichever_way_its_strides_are_written(fake, batch, seqlen, heads):
    """Contiguous rows may be written as three zeros or in numbers, and a dimension
    with one entry may carry any stride: the output is q itself all the same."""
    numbers = [seqlen * heads * 64 if batch > 1 else 7, heads * 64 if seqlen > 1 else 7, 64 if heads > 1 else 7]
    for si, so in ((numbers, (0, 0, 0)), ((0, 0, 0), numbers), (numbers, numbers)):
        fake.fake_reset(-1)
        p = rope_params(batch=batch, seqlen=seqlen, nhead_q=heads, nhead_kv=0, q=A[1], q_out=A[1], stride_q=si, stride_q_out=so)
        assert fake.attn_rope(ctypes.byref(p), None) == 0, (si, so)
        assert fake.fake_done() == 1
