// attn_kv_weigh for long query segments, on tcgen05 tensor cores.
//
// A CTA owns 128 keys of one request and kv head: their e4m3 bytes become a 16-bit
// tile in shared memory once (exactly, in the type of q), and all query rows that see
// any of them pass by:
//
//   S^T = K Q^T            (M = 128 keys, N = query rows, token x head of the group)
//   w_j += sum over columns of exp2(s log2(e) 2^ek S^T - log2(e) LSE)
//
// With the keys on the TMEM lanes a thread owns one key: its scale is a register, its
// sum never leaves the thread, and there is neither a maximum nor a second product.
// Per 128 x 128 tile of depth 128 the products take 512 clocks of the tensor cores and
// the exponentials as long (32 a clock and SM); S^T is double-buffered in TMEM, and two
// CTAs share an SM, so that one's prologue runs under the other's tiles.
//
// Where there are few key tiles, a cluster of CTAs shares one: each takes every S-th
// query tile, and the sums are added in the order of the ranks.
//
// Warps: 0-7 the exponentials (two per 32 keys, half of the columns each), 8 lane 0 loads
// query tiles (TMA), 9 owns TMEM and lane 0 issues the products, 10 keeps the query rows'
// LSE a few tiles ahead.  Every wait is bounded; where one runs out the keys' weights are NaN and the
// status says so.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "kv_weigh.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace kvweigh {

using namespace ptx;

constexpr int KM = 128;                 // keys of a CTA
constexpr int EXP_WARPS = 8;            // two per 32 keys, half of the query rows each
constexpr int LOAD_WARP = 8, MMA_WARP = 9, LSE_WARP = 10;
constexpr int TC_THREADS = 32 * 11;
constexpr int COL_RING = 4;             // query tiles whose LSE are held
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;

template <int DQK>
struct TcCfg {
  static constexpr int N = DQK <= 128 ? 128 : 64;      // query rows of a tile
  static constexpr int NCH = DQK / 64;
  static constexpr int ST = DQK == 64 ? 4 : 2;         // query tiles in flight
  static constexpr int KCH = KM * 128, QCH = N * 128;  // a 64-column chunk
  static constexpr int OFF_Q = NCH * KCH;
  static constexpr int OFF_NL = OFF_Q + ST * NCH * QCH;      // float[COL_RING][N]: -LSE in log2 units
  static constexpr int OFF_TOK = OFF_NL + COL_RING * N * 4;  // int[N]: token of a row in its tile
  static constexpr int OFF_SUM = OFF_TOK + N * 4;            // float[2][KM]: halves of the sums
  static constexpr int OFF_ODD = OFF_SUM + 2 * KM * 4;           // int[COL_RING]: a row adds nothing
  static constexpr int NBAR = 2 * ST + 4 + 2 * COL_RING + 1;
  static constexpr int OFF_BAR = OFF_ODD + COL_RING * 4;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;         // + alignment slack
  // two CTAs per SM at most: more would wait for TMEM
  static constexpr int SMEM = BYTES > 80 * 1024 ? BYTES : 80 * 1024;
  static constexpr uint32_t TMEM = 2 * N;
  enum { Q_FULL = 0, Q_EMPTY = ST, S_FULL = 2 * ST, S_EMPTY = S_FULL + 2, C_FULL = S_EMPTY + 2, C_EMPTY = C_FULL + COL_RING,
         DRAIN = C_EMPTY + COL_RING };
  static_assert(OFF_BAR % 8 == 0 && SMEM <= 232448, "layout");
};

struct TcArgs {
  Args a;
  int tok;                // query tokens of a tile: N / g
  int tiles;              // key tiles of max_k keys
  int share;              // CTAs that share a key tile
};

struct TcCtx {
  uint64_t* bar;
  volatile int* stop;
};
__device__ __noinline__ bool tc_wait_slow(const TcCtx& c, uint32_t a, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_sleep(a, parity, 20000)) {
    if (*c.stop) return false;
    if (globaltimer() - t0 > WAIT_LIMIT_NS) {
      *c.stop = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool tc_wait(const TcCtx& c, int i, uint32_t parity) {
  const uint32_t a = smem_u32(c.bar + i);
  return mbar_test_wait(a, parity) || tc_wait_slow(c, a, parity);
}
__device__ __forceinline__ bool tc_wait_warp(const TcCtx& c, int i, uint32_t parity) {
  return __all_sync(0xffffffffu, tc_wait(c, i, parity));
}

// Two e4m3 values in 16 bits each, exactly.
__device__ __forceinline__ uint32_t widen2(uint16_t x, __half*) { return e4m3x2_to_h2(x); }
__device__ __forceinline__ uint32_t widen2(uint16_t x, __nv_bfloat16*) {
  const uint32_t h = e4m3x2_to_h2(x);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);   // their upper halves
}

// The float at p of CTA `rank`'s shared memory.
__device__ __forceinline__ float peek(const float* p, int rank) {
  float x;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(x) : "r"(smem_u32(p)), "r"(rank) : "memory");
  return x;
}

template <int DQK, typename T>
__global__ void __launch_bounds__(TC_THREADS, 2) weigh_tc_kernel(const __grid_constant__ CUtensorMap q_map, const TcArgs X) {
  using C = TcCfg<DQK>;
  const Args& A = X.a;
  // block -> (request, kv head, key tile, share): the first key tiles, which see the
  // most queries, first
  const int rank = blockIdx.x % X.share, item = blockIdx.x / X.share;
  const int jobs = gridDim.x / X.share / X.tiles, kt = item / jobs, job = item - kt * jobs;
  const int b = job / A.c.hkv, hk = job - b * A.c.hkv;
  const Segment J = segment_of(A, b);
  // All returns below are the same for the whole cluster, and wait for the short
  // segments' kernel: this one is not complete before it.
  auto done = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  if (J.lq <= A.long_from) return done();     // the other kernel's, or none
  const MaskArgs mk = mask_args(A.mask, A.left, A.right, J.lq, J.lk);
  int kfrom, kto;
  seen_by(mk, J.lk, 0, J.lq - 1, kfrom, kto);
  if (A.decay != 1.f) kfrom = 0, kto = J.lk - 1;
  const int key0 = (kfrom / KM + kt) * KM;
  if (kfrom > kto || key0 > kto) return done();
  const int key1 = min(key0 + KM - 1, J.lk - 1);
  // query tiles with a row that sees one of the keys
  long long i_lo = 0, i_hi = J.lq - 1;
  if (mk.right >= 0) i_lo = max(i_lo, (long long)key0 - mk.off - mk.right);
  if (mk.left >= 0) i_hi = min(i_hi, (long long)key1 - mk.off + mk.left);
  const int qt0 = i_lo <= i_hi ? (int)(i_lo / X.tok) : 0;
  const int all = i_lo <= i_hi ? (int)(i_hi / X.tok) - qt0 + 1 : 0;
  const int n = all > rank ? (all - rank + X.share - 1) / X.share : 0;     // of this CTA

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // the swizzle counts from 1024
  float* s_nl = reinterpret_cast<float*>(smem + C::OFF_NL);
  int* s_tok = reinterpret_cast<int*>(smem + C::OFF_TOK);
  float* s_sum = reinterpret_cast<float*>(smem + C::OFF_SUM);
  int* s_odd = reinterpret_cast<int*>(smem + C::OFF_ODD);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* stop = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
  const TcCtx ctx{bar, stop}, own{bar, stop + 1};   // own: what this CTA has in flight, waited for in any case
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int used = X.tok * A.g;               // rows of a tile that are loaded
  if (tid == 0) {
    stop[0] = stop[1] = 0;
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(bar + C::Q_FULL + i, 1);
      mbar_init(bar + C::Q_EMPTY + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + C::S_FULL + i, 1);
      mbar_init(bar + C::S_EMPTY + i, EXP_WARPS);
    }
    for (int i = 0; i < COL_RING; ++i) {
      mbar_init(bar + C::C_FULL + i, 32);
      mbar_init(bar + C::C_EMPTY + i, EXP_WARPS);
    }
    mbar_init(bar + C::DRAIN, 1);
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_holder, C::TMEM);
    tmem_relinquish();
  }
  // query rows that no load writes stay zero
  for (int i = tid; i < C::ST * C::NCH * (C::N - used) * 8; i += TC_THREADS) {
    const int chunk = i / ((C::N - used) * 8), at = i - chunk * (C::N - used) * 8;
    *reinterpret_cast<uint4*>(smem + C::OFF_Q + chunk * C::QCH + used * 128 + at * 16) = make_uint4(0, 0, 0, 0);
  }
  for (int i = tid; i < C::N; i += TC_THREADS) s_tok[i] = i / A.g;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  auto load_tile = [&](int j) {               // query tile j of this CTA
    const int s = j % C::ST;
    mbar_arrive_expect_tx(bar + C::Q_FULL + s, C::NCH * 128 * used);
    const int row = J.q0 + (qt0 + rank + j * X.share) * X.tok;
    for (int c = 0; c < C::NCH; ++c)
      tma_load_3d(smem + C::OFF_Q + (s * C::NCH + c) * C::QCH, &q_map, bar + C::Q_FULL + s, c * 64, hk * A.g, row);
  };
  if (warp == LOAD_WARP && lane == 0)
    for (int j = 0; j < min(n, C::ST); ++j) load_tile(j);

  // the keys in 16 bits: 16 bytes become two swizzled pieces of 16; rows past the
  // keys, and those of a page outside the cache, are zero
  const int shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int* table = A.table + b * A.table_stride;
  auto page_of = [&](int key) {
    const int p = __ldg(table + (key >> shift));
    return p >= 0 && p < A.c.num_pages ? p : -1;
  };
  if (n > 0) {
    constexpr int PIECES = DQK / 16;
    constexpr int HELD = 4;
    for (int i0 = tid; i0 < KM * PIECES; i0 += TC_THREADS * HELD) {
      uint4 x[HELD];
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        const int i = i0 + k * TC_THREADS, r = i / PIECES, c = i - r * PIECES;
        x[k] = make_uint4(0, 0, 0, 0);
        if (r < KM && key0 + r <= key1) {
          const int page = page_of(key0 + r);
          if (page >= 0)
            x[k] = __ldg(reinterpret_cast<const uint4*>(A.c.k + page * A.c.sk.p + ((key0 + r) & in_page) * A.c.sk.r +
                                                        hk * A.c.sk.h + c * 16));
        }
      }
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        const int i = i0 + k * TC_THREADS, r = i / PIECES, c = i - r * PIECES;
        if (r >= KM) continue;
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t y[8];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          y[2 * m] = widen2((uint16_t)w[m], (T*)nullptr);
          y[2 * m + 1] = widen2((uint16_t)(w[m] >> 16), (T*)nullptr);
        }
        uint8_t* at = smem + (c >> 2) * C::KCH + r * 128;
        const int p = (c & 3) * 2, sw = r & 7;
        *reinterpret_cast<uint4*>(at + ((p ^ sw) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(at + (((p + 1) ^ sw) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    fence_proxy_async_smem();
  }
  __syncthreads();

  if (warp == LOAD_WARP) {
    if (lane == 0) {
      int j = C::ST;
      for (; j < n; ++j) {
        if (!tc_wait(ctx, C::Q_EMPTY + j % C::ST, ((j / C::ST) & 1) ^ 1)) break;
        load_tile(j);
      }
      // no copy may still be writing this CTA's shared memory when it exits
      j = min(j, n);
      for (int i = j - 1; i >= 0 && i >= j - C::ST; --i) tc_wait(own, C::Q_FULL + i % C::ST, (i / C::ST) & 1);
    }
  } else if (warp == MMA_WARP) {
    if (lane == 0) {
      constexpr bool F16 = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t ID = idesc_f16(KM, C::N, false, false, F16);
      const uint64_t dk = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dq = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
      for (int j = 0; j < n; ++j) {
        const int s = j % C::ST, sb = j & 1;
        if (!tc_wait(ctx, C::Q_FULL + s, (j / C::ST) & 1)) break;
        if (!tc_wait(ctx, C::S_EMPTY + sb, ((j >> 1) & 1) ^ 1)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < DQK / 16; ++ks) {
          const uint32_t ok = (ks >> 2) * C::KCH + (ks & 3) * 32;
          const uint32_t oq = (s * C::NCH + (ks >> 2)) * C::QCH + (ks & 3) * 32;
          umma_ss(tmem + sb * C::N, dk + (ok >> 4), dq + (oq >> 4), ID, ks > 0 ? 1u : 0u);
        }
        umma_commit(bar + C::S_FULL + sb);
        umma_commit(bar + C::Q_EMPTY + s);
      }
      // no product may be in flight when TMEM is released
      umma_commit(bar + C::DRAIN);
      tc_wait(own, C::DRAIN, 0);
    }
  } else if (warp == LSE_WARP) {
    // rows lane, lane + 32, ... of a tile; all loads of a tile are under way together,
    // a tile ahead of their use
    int tok[C::N / 32];
    const float* head[C::N / 32];
#pragma unroll
    for (int k = 0; k < C::N / 32; ++k) {
      const int r = k * 32 + lane;
      tok[k] = s_tok[r];
      head[k] = A.lse + (long long)(hk * A.g + r - tok[k] * A.g) * A.total_q + J.q0;
    }
    float l[C::N / 32];
    auto load = [&](int j) {
      const int i0 = (qt0 + rank + j * X.share) * X.tok;
#pragma unroll
      for (int k = 0; k < C::N / 32; ++k) {
        const bool in = k * 32 + lane < used && i0 + tok[k] < J.lq;
        const float v = __ldg(in ? head[k] + i0 + tok[k] : A.lse);
        l[k] = in ? v : INFINITY;
      }
    };
    if (n > 0) load(0);
    for (int j = 0; j < n; ++j) {
      const int s = j % COL_RING;
      float nl[C::N / 32];
      bool odd = false;
#pragma unroll
      for (int k = 0; k < C::N / 32; ++k) {
        nl[k] = fabsf(l[k]) < INFINITY ? -l[k] * 1.4426950408889634f : -INFINITY;
        odd |= k * 32 + lane < used && nl[k] == -INFINITY;
      }
      if (j + 1 < n) load(j + 1);
      if (!tc_wait_warp(ctx, C::C_EMPTY + s, ((j / COL_RING) & 1) ^ 1)) break;
#pragma unroll
      for (int k = 0; k < C::N / 32; ++k) s_nl[s * C::N + k * 32 + lane] = nl[k];
      const bool any = __any_sync(0xffffffffu, odd);
      if (lane == 0) s_odd[s] = any;
      mbar_arrive(bar + C::C_FULL + s);
    }
  } else {
    // ------------------------------------------------------- exponentials
    const int half = warp >> 2, r = (warp & 3) * 32 + lane, key = key0 + r;
    constexpr int COLS = C::N / 2;
    const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * COLS;
    int page = -1;                            // of this thread's key, if its weight changes
    if (key >= kfrom && key <= kto) {
      page = page_of(key);
      if (page < 0) report(A, ATTN_ERR_BAD_PAGE);
    }
    const float u = page >= 0 ? A.scale_log2 * exp2_int(kv_exp_of(__ldg(A.c.k_exp + (long long)page * A.c.hkv + hk))) : 0.f;
    // tiles whose first token is at least need0 and whose last one is at most need1 see all keys
    const int need0 = mk.right >= 0 ? (int)max(0ll, (long long)key1 - mk.off - mk.right) : 0;
    const int need1 = mk.left >= 0 ? (int)min((long long)INT32_MAX, (long long)key0 - mk.off + mk.left) : INT32_MAX;
    // tokens that see this thread's key
    const long long see0 = mk.right >= 0 ? (long long)key - mk.off - mk.right : INT32_MIN;
    const long long see1 = mk.left >= 0 ? (long long)key - mk.off + mk.left : INT32_MAX;
    const float2 u2 = make_float2(u, u), one2 = make_float2(1.f, 1.f);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    bool ok = true;
    int i0 = (qt0 + rank) * X.tok;
    for (int j = 0; j < n; ++j, i0 += X.share * X.tok) {
      const int sb = j & 1, s = j % COL_RING;
      if (!(ok = tc_wait_warp(ctx, C::C_FULL + s, (j / COL_RING) & 1))) break;
      if (!(ok = tc_wait_warp(ctx, C::S_FULL + sb, (j >> 1) & 1))) break;
      tc_fence_after();
      // columns of this warp whose tokens see this thread's key (tokens ascend with the column)
      const int from = (int)min((long long)C::N, max(0ll, see0 - i0) * A.g) - half * COLS;
      const int to = (int)min((long long)C::N, max(0ll, see1 - i0 + 1) * A.g) - half * COLS;
      const bool plain = !s_odd[s] && i0 >= need0 && min(i0 + X.tok, J.lq) - 1 <= need1;
      const float* nl = s_nl + s * C::N + half * COLS;
#pragma unroll
      for (int c = 0; c < COLS; c += 32) {
        uint32_t v[32];
        tmem_ld32(mine + sb * C::N + c, v);
        tmem_wait_ld();
        if (c + 32 == COLS) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar + C::S_EMPTY + sb);
        }
        if (plain) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 l = *reinterpret_cast<const float4*>(nl + c + k);
            const float2 x = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), u2, make_float2(l.x, l.y));
            const float2 y = fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), u2, make_float2(l.z, l.w));
            sum[0] = fma2(make_float2(fast_exp2(x.x), fast_exp2(x.y)), one2, sum[0]);
            sum[1] = fma2(make_float2(fast_exp2(y.x), fast_exp2(y.y)), one2, sum[1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float l = nl[c + k];
            const bool adds = l > -INFINITY && c + k >= from && c + k < to;
            const float p = fast_exp2(fmaf(__uint_as_float(v[k]), u, l));
            (k & 1 ? sum[(k >> 1) & 1].y : sum[(k >> 1) & 1].x) += adds ? p : 0.f;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + C::C_EMPTY + s);
    }
    ok = __all_sync(0xffffffffu, ok);
    float w = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    if (!ok) {
      w = __int_as_float(0x7fc00000);
      if (lane == 0) report(A, ATTN_ERR_TIMEOUT);
    }
    s_sum[half * KM + r] = w;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, C::TMEM);
  }
  if (X.share > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && tid < KM) {
    const int key = key0 + tid;
    float w = s_sum[tid] + s_sum[KM + tid];
    for (int s = 1; s < X.share; ++s) w += peek(s_sum + tid, s) + peek(s_sum + KM + tid, s);
    const int page = key >= kfrom && key <= kto ? page_of(key) : -1;
    if (page >= 0) {
      const long long at = ((long long)page * A.c.hkv + hk) * (in_page + 1) + (key & in_page);
      const bool fresh = A.fresh && key >= J.lk - J.lq;
      A.weight[at] = (fresh || A.decay == 0.f ? 0.f : A.decay * A.weight[at]) + w;
      if (fresh) A.position[at] = (int)((unsigned)key + (A.offsets ? (unsigned)__ldg(A.offsets + b) : 0u));
    }
  }
  // no CTA leaves while another reads its shared memory
  if (X.share > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  done();
}

// -------------------------------------------------------------------- host

static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

template <int DQK, typename T>
static int launch_tc(const Args& a, int batch, cudaStream_t st) {
  using C = TcCfg<DQK>;
  TcArgs x{};
  x.a = a;
  x.tok = C::N / a.g;
  x.tiles = cdiv(a.max_k, KM) + 1;            // a window may begin inside a tile
  const long long items = (long long)batch * a.c.hkv * x.tiles;
  x.share = 1;
  while (x.share < 8 && items * x.share * 2 <= 2 * SMS) x.share *= 2;
  if (items * x.share > (1LL << 30)) return ATTN_ERR_INVALID_ARG;
  const auto fn = encoder();
  if (!fn) return ATTN_ERR_CUDA;
  CUtensorMap map;
  const cuuint64_t dims[3] = {(cuuint64_t)DQK, (cuuint64_t)a.hq, (cuuint64_t)a.total_q};
  const cuuint64_t strides[2] = {(cuuint64_t)a.sq.h * 2, (cuuint64_t)a.sq.r * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)x.tok}, one[3] = {1, 1, 1};
  if (fn(&map, sizeof(T) == 2 && std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
         3, const_cast<void*>(a.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return ATTN_ERR_CUDA;
  const auto kern = weigh_tc_kernel<DQK, T>;
  if (!succeeded(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM))) return ATTN_ERR_CUDA;
  // It starts beside the short segments' kernel: neither touches what the other does, and
  // that one began after all earlier work.
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = x.share;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * x.share));
  cfg.blockDim = dim3(TC_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return succeeded(cudaLaunchKernelEx(&cfg, kern, map, x)) ? ATTN_OK : ATTN_ERR_CUDA;
}

template <typename T>
static int launch_tc(const Args& a, int dqk, int batch, cudaStream_t st) {
  if (dqk == 64) return launch_tc<64, T>(a, batch, st);
  if (dqk == 128) return launch_tc<128, T>(a, batch, st);
  if (dqk == 192) return launch_tc<192, T>(a, batch, st);
  return launch_tc<256, T>(a, batch, st);
}

int long_group(int dqk) { return dqk <= 128 ? 128 : 64; }

int launch_long(const Args& a, bool bf16, int dqk, int batch, cudaStream_t st) {
  return bf16 ? launch_tc<__nv_bfloat16>(a, dqk, batch, st) : launch_tc<__half>(a, dqk, batch, st);
}

}  // namespace kvweigh
}  // namespace attn
