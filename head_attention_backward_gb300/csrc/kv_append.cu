// New keys and values quantised into the paged cache (attn_kv_append): e4m3
// values under one power-of-two scale per page, kv head and side.
//
// Memory bound (2 bytes read and 1 written per value).  The unit of work is a
// run (the new tokens of one page) of one head and side, because the scale
// needs the run's largest magnitude before the first value can be written.  A
// group of 1 to 8 warps owns it, enough to hold a full page of values in
// registers between the two passes (up to 16,384 values; more are read twice).
#include "common.cuh"
#include "kv_common.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace kvappend {

constexpr int NWARPS = 8;
constexpr int RESIDENT = 3;   // CTAs per SM that the registers have to allow
constexpr int NTHREADS = 32 * NWARPS;
constexpr int HELD = 8;   // 16-byte pieces of a run that a lane keeps in registers

struct Args {
  const void* k;
  const void* v;
  Strides sk, sv;
  const int64_t* slots;
  int tokens, tile;
  int gw;              // warps of a group: 1, 2, 4 or 8
  KvCacheView c;
};

constexpr int MAX_RUN = 256;   // tokens of a run: the largest page

// The new tokens of one page, and their rows in it: token t + i in row first +
// i, or by a list in shared memory where they are not in order.
struct Run {
  int t, n, first;   // first: the least row
  const int* tok;
  const uint8_t* at;
};

__device__ __forceinline__ float2 up2(uint32_t x, __nv_bfloat16*) {
  // a bf16 is the upper half of an fp32
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float2 up2(uint32_t x, __half*) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }

// Larger finite magnitudes of two pairs.  |x| + 0 |x| is |x| where x is finite and
// NaN elsewhere, which the maximum passes over.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t x, __nv_bfloat16*) {
  x &= 0x7fff7fffu;
  const __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&x);
  const __nv_bfloat162 y = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&m), __hfma2(v, __float2bfloat162_rn(0.f), v));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t x, __half*) {
  x &= 0x7fff7fffu;
  const __half2 v = *reinterpret_cast<__half2*>(&x);
  const __half2 y = __hmax2(*reinterpret_cast<__half2*>(&m), __hfma2(v, __float2half2_rn(0.f), v));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from amax's exponent and
// mantissa; limited to the format's range (a subnormal or zero amax is far
// below it).
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < KV_EXP_MIN ? KV_EXP_MIN : e > KV_EXP_MAX ? KV_EXP_MAX : e;
}

template <typename T>
__device__ __forceinline__ uint32_t amax8(uint32_t m, const uint4& x) {
  m = amax2(m, x.x, (T*)nullptr);
  m = amax2(m, x.y, (T*)nullptr);
  m = amax2(m, x.z, (T*)nullptr);
  return amax2(m, x.w, (T*)nullptr);
}

// 8 values over 2^e as e4m3.  bf16: the product with a power of two is exact
// in bf16 (values that leave its range are 0 in e4m3 anyway).  fp16: likewise
// while the factor is one of its normal numbers -- what becomes subnormal is
// below 2^-14, far under half of e4m3's least value -- else in fp32.
struct Quantiser {
  uint32_t factor;     // 2^-e twice in the input type, or 0: use inv
  float inv;           // 2^-e
};
__device__ __forceinline__ Quantiser quantiser(int e, __nv_bfloat16*) {
  const __nv_bfloat162 f = __float2bfloat162_rn(exp2_int(-e));
  return {*reinterpret_cast<const uint32_t*>(&f), exp2_int(-e)};
}
__device__ __forceinline__ Quantiser quantiser(int e, __half*) {
  const __half2 f = __float2half2_rn(exp2_int(-e));
  return {e >= -14 && e <= 14 ? *reinterpret_cast<const uint32_t*>(&f) : 0u, exp2_int(-e)};
}
__device__ __forceinline__ uint32_t quantise2(uint32_t x, const Quantiser& q, __nv_bfloat16*) {
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&q.factor));
  const float2 f = up2(*reinterpret_cast<const uint32_t*>(&y), (__nv_bfloat16*)nullptr);
  return f2_to_e4m3x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t quantise2(uint32_t x, const Quantiser& q, __half*) {
  if (q.factor) {
    const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<const __half2*>(&q.factor));
    return h2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&y));
  }
  const float2 f = up2(x, (__half*)nullptr);
  return f2_to_e4m3x2(f.x * q.inv, f.y * q.inv);
}
template <typename T>
__device__ __forceinline__ uint2 quantise8(const uint4& x, const Quantiser& q) {
  T* t = nullptr;
  return make_uint2(__byte_perm(quantise2(x.x, q, t), quantise2(x.y, q, t), 0x5410),
                    __byte_perm(quantise2(x.z, q, t), quantise2(x.w, q, t), 0x5410));
}

template <int N> struct Dim { static constexpr int value = N; };

// The threads that share a run.
struct Group {
  int id, n, tid;      // of the CTA's groups; threads; this thread's place
  __device__ __forceinline__ void sync() const {
    if (n == 32) __syncwarp();
    else ptx::named_bar_sync(1 + id, n);
  }
};

// The live rows in front of a run at a larger scale (f: old over new), 16 values
// at a time.
template <int D>
__device__ __noinline__ void round_again(int rows, uint8_t* cache, long long cr, float f, int tid, int n) {
  for (int i = tid; i < rows * (D / 16); i += n) {
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

// What both forms below do between the passes: the run's scale from the
// threads' largest magnitudes, and the rows in front of the run.
template <typename T, int D>
__device__ __forceinline__ int settle_scale(const Run& r, uint32_t m, uint8_t* cache, long long cr, uint8_t* exp_byte,
                                            int old, const Group& G, uint32_t* red) {
  // magnitudes order like their bits
  const float2 mm = up2(m, (T*)nullptr);
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mm.x, mm.y)));
  if (G.n > 32) {
    if ((G.tid & 31) == 0) red[G.tid >> 5] = top;
    G.sync();   // also: every thread has read the old scale
    for (int w = 0; w < G.n / 32; ++w) top = max(top, red[w]);
  }
  const int e = max(old, exponent_of(__uint_as_float(top)));
  if (r.first > 0 && e > old) round_again<D>(r.first, cache, cr, exp2_int(old - e), G.tid, G.n);
  if (G.tid == 0) *exp_byte = (uint8_t)(e + KV_EXP_BIAS);
  return e;
}

// How a group covers a run: a thread keeps to one piece of 8 columns and takes
// every step-th row.
template <int D>
struct Cover {
  int row, step, col;
  __device__ __forceinline__ explicit Cover(const Group& G) {
    constexpr int PER = D / 8;
    step = G.n / PER;
    row = G.tid / PER;
    col = G.tid % PER * 8;
    if (row >= step) row = 1 << 16;   // left over where PER is no power of two: no row
  }
};

// One run of one head and side, by one group, its tokens in order: in blocks of
// what the group can hold, the last of which (as a rule the only one) stays in
// registers.  red: a word per warp of the group, not the last item's.
template <typename T, int D>
__device__ __forceinline__ void append_in_order(const Run& r, const T* x, long long xr, uint8_t* cache, long long cr,
                                                uint8_t* exp_byte, const Group& G, uint32_t* red) {
  const Cover<D> c(G);
  const int old = r.first > 0 ? kv_exp_of(*exp_byte) : KV_EXP_MIN;
  const long long sstep = c.step * xr, dstep = c.step * cr;
  uint4 held[HELD];
  auto load = [&](int row) {     // rows row, row + step, ...
    const T* src = x + (r.t + row) * xr + c.col;
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      held[k] = make_uint4(0, 0, 0, 0);
      if (row + c.step * k < r.n) held[k] = __ldg(reinterpret_cast<const uint4*>(src));
      src += sstep;
    }
  };
  uint32_t m = 0;
  const int last = (r.n - 1) / (HELD * c.step);      // blocks before the last one
  int row = c.row;
  for (int i = 0;; ++i) {
    load(row);
#pragma unroll
    for (int k = 0; k < HELD; ++k) m = amax8<T>(m, held[k]);
    if (i == last) break;
    row += HELD * c.step;
  }
  const Quantiser q = quantiser(settle_scale<T, D>(r, m, cache, cr, exp_byte, old, G, red), (T*)nullptr);
  for (int i = last;; --i) {
    uint8_t* dst = cache + (r.first + row) * cr + c.col;
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      if (row + c.step * k < r.n) *reinterpret_cast<uint2*>(dst) = quantise8<T>(held[k], q);
      dst += dstep;
    }
    if (i == 0) break;
    row -= HELD * c.step;
    load(row);
  }
}

// A run whose tokens are not in order, by its list; the values are read twice.
template <typename T, int D>
__device__ __noinline__ void append_listed(const Run& r, const T* x, long long xr, uint8_t* cache, long long cr,
                                        uint8_t* exp_byte, const Group& G, uint32_t* red) {
  const Cover<D> c(G);
  auto load = [&](int row) {
    return __ldg(reinterpret_cast<const uint4*>(x + (long long)r.tok[row] * xr + c.col));
  };
  const int old = r.first > 0 ? kv_exp_of(*exp_byte) : KV_EXP_MIN;
  uint32_t m = 0;
#pragma unroll 8
  for (int row = c.row; row < r.n; row += c.step) m = amax8<T>(m, load(row));
  const Quantiser q = quantiser(settle_scale<T, D>(r, m, cache, cr, exp_byte, old, G, red), (T*)nullptr);
#pragma unroll 8
  for (int row = c.row; row < r.n; row += c.step) {
    *reinterpret_cast<uint2*>(cache + (long long)r.at[row] * cr + c.col) = quantise8<T>(load(row), q);
  }
}

// A CTA takes the runs that start in its tile of tokens (at most 32), and of
// each the heads and sides of its share (blockIdx.y), one per group at a time.
// A run is found by its page: it starts at a token whose page none of the
// page_size tokens before it has, and ends where page_size tokens in a row
// have another.
template <typename T, int DQK, int DV>
__global__ void __launch_bounds__(NTHREADS, RESIDENT) append_kernel(const Args A) {
  __shared__ int s_tok[NWARPS][MAX_RUN];       // a list per group
  __shared__ uint8_t s_at[NWARPS][MAX_RUN];
  __shared__ int2 s_run[NWARPS];
  __shared__ uint32_t s_red[2 * NWARPS];
  const int lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * A.tile;
  const int shift = A.c.page_shift, size = 1 << shift;
  const long long limit = (long long)A.c.num_pages << shift;
  // a load without a branch, so that many are on their way together (pages of 128:
  // 8.2 us against 9.4)
  auto slot_at = [&](int t) -> long long {
    const bool in = t >= 0 && t < A.tokens;
    const long long s = (long long)__ldg(A.slots + (in ? t : t0));
    return in && s < limit ? s : -1;
  };
  auto page_at = [&](int t) {   // -1: none
    const long long s = slot_at(t);
    return s < 0 ? -1 : (int)(s >> shift);
  };
  const int mine = lane < A.tile ? page_at(t0 + lane) : -1;
  uint32_t maybe = __ballot_sync(0xffffffffu, mine >= 0 && mine != page_at(t0 + lane - 1));
  Group G;
  G.n = 32 * A.gw;
  G.id = threadIdx.x / G.n;
  G.tid = threadIdx.x % G.n;
  const int groups = NWARPS / A.gw, share = groups * gridDim.y;   // groups at work on one run
  const int per_run = A.c.hkv * 2;
  int turn = 0;
  for (; maybe; maybe &= maybe - 1) {
    const int l = __ffs(maybe) - 1, t = t0 + l;
    const long long slot = slot_at(t);
    const int page = (int)(slot >> shift), row = (int)(slot & (size - 1));
    // the tokens before, and those up to 2 page_size on, without a wait between:
    // whether an earlier one has the page; the run's length if it is in order;
    // whether the page comes again after that
    bool earlier = false;
#pragma unroll 2
    for (int j = 2 + lane; j <= size; j += 32) earlier |= page_at(t - j) == page;
    int n = size - row;
    bool again = false;
    for (int base = 0; base < 2 * size; base += 128) {
      long long s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = base + 32 * k < 2 * size ? slot_at(t + base + 32 * k + lane) : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = base + 32 * k + lane;
        const uint32_t stop = __ballot_sync(0xffffffffu, i < n && s[k] != slot + i);
        if (stop) n = base + 32 * k + __ffs(stop) - 1;
        again |= i >= n && i < n + size && s[k] >= 0 && (int)(s[k] >> shift) == page;
      }
    }
    if (__any_sync(0xffffffffu, earlier)) continue;
    Run r{t, n, row, nullptr, nullptr};
    int hs = blockIdx.y * groups + G.id;
    if (hs >= per_run) continue;
    const bool list = __any_sync(0xffffffffu, again);
    if (list) {
      G.sync();                     // the last list has been used
      if (G.tid < 32) {
        int count = 0, first = size, last = t;
        for (int base = t; count < size && base < A.tokens && base - last <= size; base += 32) {
          const long long s = slot_at(base + lane);
          const bool same = s >= 0 && (int)(s >> shift) == page;
          const uint32_t all = __ballot_sync(0xffffffffu, same);
          const int at = count + __popc(all & ((1u << lane) - 1));
          if (same && at < size) {
            s_tok[G.id][at] = base + lane;
            s_at[G.id][at] = (uint8_t)(s & (size - 1));
            first = min(first, (int)(s & (size - 1)));
          }
          if (all) last = base + 31 - __clz(all);
          count = min(size, count + __popc(all));
        }
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) s_run[G.id] = make_int2(count, first);
      }
      G.sync();
      r = Run{t, s_run[G.id].x, s_run[G.id].y, s_tok[G.id], s_at[G.id]};
    }
    for (; hs < per_run; hs += share) {
      turn ^= NWARPS;
      const int h = hs >> 1;
      const bool is_v = hs & 1;
      uint8_t* exp_byte = (is_v ? A.c.v_exp : A.c.k_exp) + (long long)page * A.c.hkv + h;
      uint8_t* cache = is_v ? A.c.v + page * A.c.sv.p + h * A.c.sv.h : A.c.k + page * A.c.sk.p + h * A.c.sk.h;
      const T* x = is_v ? static_cast<const T*>(A.v) + h * A.sv.h : static_cast<const T*>(A.k) + h * A.sk.h;
      const long long xr = is_v ? A.sv.r : A.sk.r, cr = is_v ? A.c.sv.r : A.c.sk.r;
      uint32_t* red = s_red + turn + G.id * A.gw;   // two sets in turn: one barrier per item
      auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (list) append_listed<T, D>(r, x, xr, cache, cr, exp_byte, G, red);
        else append_in_order<T, D>(r, x, xr, cache, cr, exp_byte, G, red);
      };
      if (DQK == DV || !is_v) go(Dim<DQK>());
      else go(Dim<DV>());
    }
  }
}

template <typename T>
static void launch(const Args& a, int dqk, int dv, dim3 grid, cudaStream_t st) {
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
  // a group holds HELD pieces of 8 values per thread: a whole page, if 8 warps can
  const int dim = p->cache.d_qk > p->cache.d_v ? p->cache.d_qk : p->cache.d_v;
  a.gw = 1;
  while (a.gw < NWARPS && HELD * (a.gw * 32 / (dim / 8)) < p->cache.page_size) a.gw *= 2;
  // Items a group takes one after the other: as many as leave the GPU full, up
  // to four, beyond which the CTAs' search for runs no longer weighs (15,295
  // tokens in pages of 64: 24.4 us at four, 27.9 at one, 32.6 at eight; 64 single
  // tokens: 4.0 us at one, 4.6 at four).
  const int groups = NWARPS / a.gw, per_run = p->cache.nhead_kv * 2;
  const long long full = (long long)(p->tokens / p->cache.page_size) * per_run / ((long long)groups * SMS * RESIDENT);
  const int rounds = full < 1 ? 1 : full > 4 ? 4 : (int)full;
  const int shares = cdiv(per_run, groups * rounds);
  // Tokens a CTA searches for runs: one in short calls (where every token may
  // start one), up to a warp's width as the grid grows.
  const long long tile = cdiv_ll((long long)p->tokens * shares, 1024);
  a.tile = tile > 32 ? 32 : (int)tile;
  const dim3 grid(cdiv(p->tokens, a.tile), shares);
  if (p->dtype == ATTN_BF16) launch<__nv_bfloat16>(a, p->cache.d_qk, p->cache.d_v, grid, st);
  else launch<__half>(a, p->cache.d_qk, p->cache.d_v, grid, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace kvappend
}  // namespace attn

extern "C" int attn_kv_append(const attn_kv_append_params* p, cudaStream_t stream) {
  return attn::kvappend::run(p, stream);
}
