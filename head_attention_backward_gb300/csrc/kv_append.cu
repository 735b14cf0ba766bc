// New keys and values quantised into the paged cache (attn_kv_append): e4m3
// values under one power-of-two scale per page, kv head and side.
//
// Memory bound (2 bytes read and 1 written per value).  The unit of work is a
// run (the new tokens of one page) of one head and side; a warp owns it,
// because the scale needs the run's largest magnitude before the first value
// can be written.  A short run stays in registers between the two passes.
#include "common.cuh"
#include "kv_common.cuh"

namespace attn {
namespace kvappend {

constexpr int NWARPS = 8;
constexpr int NTHREADS = 32 * NWARPS;
constexpr int HELD = 8;   // 16-byte pieces of a run that a lane keeps in registers

struct Args {
  const void* k;
  const void* v;
  Strides sk, sv;
  const int64_t* slots;
  int tokens, tile;
  KvCacheView c;
};

constexpr int MAX_RUN = 256;   // tokens of a run: the largest page

// The new tokens of one page, and their rows in it (in shared memory).
struct Run {
  const int* tok;
  const uint8_t* at;
  int n, first;      // tokens; least row among them
};

__device__ __forceinline__ float2 up2(uint32_t x, __nv_bfloat16*) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x));
}
__device__ __forceinline__ float2 up2(uint32_t x, __half*) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }

// Least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from amax's exponent and
// mantissa; limited to the format's range (a subnormal or zero amax is far
// below it).
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < KV_EXP_MIN ? KV_EXP_MIN : e > KV_EXP_MAX ? KV_EXP_MAX : e;
}

template <typename T>
__device__ __forceinline__ float amax8(float m, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = up2(w[i], (T*)nullptr);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));   // a NaN is passed over
  }
  return m;
}

template <typename T>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = up2(w[i], (T*)nullptr);
    q[i] = f2_to_e4m3x2(f.x * inv, f.y * inv);
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// One run of one head and side, by one warp.  D: head dim.
template <typename T, int D>
__device__ __forceinline__ void append_run(const Run& r, const T* x, long long xr, uint8_t* cache, long long cr,
                                           uint8_t* exp_byte, int lane) {
  constexpr int PER = D / 8;   // pieces of 8 values per row
  const int pieces = r.n * PER;
  auto load = [&](int i) {
    return __ldg(reinterpret_cast<const uint4*>(x + (long long)r.tok[i / PER] * xr + (i % PER) * 8));
  };
  const int old = r.first > 0 ? kv_exp_of(*exp_byte) : KV_EXP_MIN;
  uint4 held[HELD];
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (lane + 32 * k < pieces) held[k] = load(lane + 32 * k);
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (lane + 32 * k < pieces) m = amax8<T>(m, held[k]);
  for (int i = lane + 32 * HELD; i < pieces; i += 32) m = amax8<T>(m, load(i));
  // magnitudes order like their bits
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  const int e = max(old, exponent_of(m));
  if (r.first > 0 && e > old) {
    // the live rows in front of the run, 16 values at a time
    const float f = exp2_int(old - e);
    for (int i = lane; i < r.first * (D / 16); i += 32) {
      uint4* at = reinterpret_cast<uint4*>(cache + (long long)(i / (D / 16)) * cr + (i % (D / 16)) * 16);
      const uint4 was = *at;
      const uint32_t w[4] = {was.x, was.y, was.z, was.w};
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = e4m3x2_to_h2((uint16_t)w[j]), hi = e4m3x2_to_h2((uint16_t)(w[j] >> 16));
        const float2 a = up2(lo, (__half*)nullptr), b = up2(hi, (__half*)nullptr);
        q[j] = f2_to_e4m3x2(a.x * f, a.y * f) | ((uint32_t)f2_to_e4m3x2(b.x * f, b.y * f) << 16);
      }
      *at = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  const float inv = exp2_int(-e);
  auto store = [&](int i, const uint4& v) {
    *reinterpret_cast<uint2*>(cache + (long long)r.at[i / PER] * cr + (i % PER) * 8) = quantise8<T>(v, inv);
  };
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (lane + 32 * k < pieces) store(lane + 32 * k, held[k]);
  for (int i = lane + 32 * HELD; i < pieces; i += 32) store(i, load(i));
  if (lane == 0) *exp_byte = (uint8_t)(e + KV_EXP_BIAS);
}

// A CTA takes the runs that start in its tile of tokens (at most 32), all
// heads and both sides of each, one (run, head, side) per warp at a time.  A
// run is found by its page: it starts at a token whose page none of the
// page_size tokens before it has, and ends where page_size tokens in a row have
// another.
template <typename T, int DQK, int DV>
__global__ void __launch_bounds__(NTHREADS) append_kernel(const Args A) {
  __shared__ int s_tok[NWARPS][MAX_RUN];
  __shared__ uint8_t s_at[NWARPS][MAX_RUN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * A.tile;
  const int shift = A.c.page_shift, size = 1 << shift;
  const long long limit = (long long)A.c.num_pages << shift;
  auto slot_at = [&](int t) -> long long {
    const long long s = t >= 0 && t < A.tokens ? (long long)__ldg(A.slots + t) : -1;
    return s < limit ? s : -1;
  };
  auto page_at = [&](int t) {   // -1: none
    const long long s = slot_at(t);
    return s < 0 ? -1 : (int)(s >> shift);
  };
  const int mine = lane < A.tile ? page_at(t0 + lane) : -1;
  uint32_t maybe = __ballot_sync(0xffffffffu, mine >= 0 && mine != page_at(t0 + lane - 1));
  uint32_t starts = 0;
  for (; maybe; maybe &= maybe - 1) {
    const int l = __ffs(maybe) - 1, page = __shfl_sync(0xffffffffu, mine, l);
    bool seen = false;
    for (int j = 2 + lane; j <= size; j += 32) seen |= page_at(t0 + l - j) == page;
    if (!__any_sync(0xffffffffu, seen)) starts |= 1u << l;
  }
  const int per_run = A.c.hkv * 2;
  const int items = __popc(starts) * per_run;
  int listed = -1;
  Run r{s_tok[warp], s_at[warp], 0, 0};
  int page = 0;
  for (int i = warp; i < items; i += NWARPS) {
    const int which = i / per_run, hs = i - which * per_run, h = hs >> 1;
    if (which != listed) {
      listed = which;
      const int t = t0 + (int)__fns(starts, 0, which + 1);
      page = page_at(t);
      int n = 0, first = size, last = t;
      __syncwarp();
      for (int base = t; n < size && base < A.tokens && base - last <= size; base += 32) {
        const long long s = slot_at(base + lane);
        const bool same = s >= 0 && (int)(s >> shift) == page;
        const uint32_t all = __ballot_sync(0xffffffffu, same);
        const int at = n + __popc(all & ((1u << lane) - 1));
        if (same && at < size) {
          s_tok[warp][at] = base + lane;
          s_at[warp][at] = (uint8_t)(s & (size - 1));
          first = min(first, (int)(s & (size - 1)));
        }
        if (all) last = base + 31 - __clz(all);
        n = min(size, n + __popc(all));
      }
      r.n = n;
      r.first = __reduce_min_sync(0xffffffffu, first);
      __syncwarp();
    }
    const long long eo = (long long)page * A.c.hkv + h;
    if ((hs & 1) == 0)
      append_run<T, DQK>(r, static_cast<const T*>(A.k) + h * A.sk.h, A.sk.r, A.c.k + page * A.c.sk.p + h * A.c.sk.h,
                         A.c.sk.r, A.c.k_exp + eo, lane);
    else
      append_run<T, DV>(r, static_cast<const T*>(A.v) + h * A.sv.h, A.sv.r, A.c.v + page * A.c.sv.p + h * A.c.sv.h,
                        A.c.sv.r, A.c.v_exp + eo, lane);
  }
}

template <typename T>
static void launch(const Args& a, int dqk, int dv, int grid, cudaStream_t st) {
  if (dqk == 64) append_kernel<T, 64, 64><<<grid, NTHREADS, 0, st>>>(a);
  else if (dqk == 128) append_kernel<T, 128, 128><<<grid, NTHREADS, 0, st>>>(a);
  else if (dqk == 192) append_kernel<T, 192, 128><<<grid, NTHREADS, 0, st>>>(a);
  else append_kernel<T, 256, 256><<<grid, NTHREADS, 0, st>>>(a);
}

static int run(const attn_kv_append_params* p, cudaStream_t st) {
  if (!p || (p->dtype != ATTN_BF16 && p->dtype != ATTN_FP16)) return ATTN_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->tokens > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  Args a{};
  const int s = kv_resolve(p->cache, &a.c);
  if (s != ATTN_OK) return s;
  if (p->tokens == 0) return ATTN_OK;
  if (!p->k || !p->v || !p->slots || !aligned_to(p->k, 16) || !aligned_to(p->v, 16) || !aligned_to(p->slots, 8))
    return ATTN_ERR_INVALID_ARG;
  if (!packed_strides(p->stride_k, p->cache.nhead_kv, p->cache.d_qk, &a.sk) ||
      !packed_strides(p->stride_v, p->cache.nhead_kv, p->cache.d_v, &a.sv))
    return ATTN_ERR_INVALID_ARG;
  a.k = p->k;
  a.v = p->v;
  a.slots = p->slots;
  a.tokens = p->tokens;
  a.tile = p->tokens <= 4096 ? 1 : 16;
  const int grid = cdiv(p->tokens, a.tile);
  if (p->dtype == ATTN_BF16) launch<__nv_bfloat16>(a, p->cache.d_qk, p->cache.d_v, grid, st);
  else launch<__half>(a, p->cache.d_qk, p->cache.d_v, grid, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace kvappend
}  // namespace attn

extern "C" int attn_kv_append(const attn_kv_append_params* p, cudaStream_t stream) {
  return attn::kvappend::run(p, stream);
}
