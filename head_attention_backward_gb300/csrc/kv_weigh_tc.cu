// attn_kv_weigh for long query segments, on tcgen05 tensor cores.
//
// A work item is 128 keys of one request and kv head: their e4m3 bytes become a 16-bit
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
// CTAs share an SM, so that one's waits run under the other's tiles: an SM takes 1,075
// clocks a tile while both are at theirs, 1,577 while one is.  Two forms that were slower
// (4 x 1,024 tokens over 5,120, this one 154 us, 890 TFLOP/s): 256 keys per item, kept in
// TMEM, one CTA per SM (198), which halves the query tiles' way through L2 and shared
// memory, but that bounds nothing; and 304 persistent CTAs that fetch the next item's keys
// while they work (186): the registers for it cost the inner loop more than an item's
// beginning (TMEM 2.4 us, keys 1.4) costs beside another CTA's tiles.
//
// The items are those of the long segments alone.  Where the bounds leave room for many,
// each CTA lists them for itself, so that a loose max_seqlen_k, or many short segments,
// cost only CTAs that find nothing left.  Where there are few, a cluster of CTAs shares
// one: each takes every S-th query tile, and the sums are added in the order of the ranks.
//
// Warps: 0-7 the exponentials (two per 32 keys, half of the columns each), 8 lane 0 loads
// query tiles (TMA), 9 owns TMEM and lane 0 issues the products, 10 keeps the query rows'
// LSE a few tiles ahead.  Every wait is bounded; where one runs out the keys' weights are
// NaN and the status says so.
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
constexpr int LIST = 256;               // segments whose items are listed at a time
// Where the bounds leave room for few items, each has a CTA, and they go by key tile: the
// first ones see the most queries, the short ones come last (16 x 1,000 tokens: 107 us, 125
// from a list, which goes by segment; 4 x 1,024 over 5,120: 154 and 158).
constexpr int MAX_PLACES = 4096;
// CTAs for a list at most.  Those beyond the 304 that reside begin as others end, which
// evens out ragged items, and pay for TMEM again, 2.4 us (8 requests of 4,000 tokens, 64
// new: 55 us with 608, 60 with 2,048).
constexpr int MAX_TC_GRID = 608;
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
  static constexpr int OFF_ODD = OFF_SUM + 2 * KM * 4;       // int[COL_RING]: a row adds nothing
  static constexpr int OFF_LIST = OFF_ODD + COL_RING * 4;    // int[LIST + 12]: key tiles before a segment of the list; of a warp's
  static constexpr int OFF_BAR = OFF_LIST + (LIST + 12) * 4;
  enum { Q_FULL = 0, Q_EMPTY = ST, S_FULL = 2 * ST, S_EMPTY = S_FULL + 2, C_FULL = S_EMPTY + 2, C_EMPTY = C_FULL + COL_RING,
         NBAR = C_EMPTY + COL_RING };
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;         // + alignment slack
  // two CTAs per SM at most: more would wait for TMEM
  static constexpr int SMEM = BYTES > 80 * 1024 ? BYTES : 80 * 1024;
  static constexpr int RESIDENT = SMEM <= 113 * 1024 ? 2 : 1;
  static constexpr uint32_t TMEM = 2 * N;
  static_assert(OFF_BAR % 8 == 0 && SMEM <= 232448, "layout");
};

struct TcArgs {
  Args a;
  int batch;
  int tok;                // query tokens of a tile: N / g
  int share;              // CTAs that share an item
  int places;             // items that the bounds leave room for, a CTA each; 0: they are listed
};

__device__ __forceinline__ void mbar_inval(uint64_t* bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct TcCtx {
  uint64_t* bar;
  volatile int* stop;
};
template <uint64_t LIMIT>
__device__ __noinline__ bool tc_wait_slow(const TcCtx& c, uint32_t a, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_sleep(a, parity, 20000)) {
    if (*c.stop) return false;
    if (globaltimer() - t0 > LIMIT) {
      *c.stop = 1;
      return false;
    }
  }
  return true;
}
template <uint64_t LIMIT = WAIT_LIMIT_NS>
__device__ __forceinline__ bool tc_wait(const TcCtx& c, int i, uint32_t parity) {
  const uint32_t a = smem_u32(c.bar + i);
  return mbar_test_wait(a, parity) || tc_wait_slow<LIMIT>(c, a, parity);
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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A long segment, and the keys of it whose weights change; kfrom > kto: none, or not a
// long segment.
struct Long {
  int q0, lq, lk, fresh, kfrom, kto;
  MaskArgs mk;
};
__device__ __forceinline__ Long long_at(const Args& A, int b) {
  Long L{};
  const Segment J = segment_of(A, b);
  L.q0 = J.q0, L.lq = J.lq, L.lk = J.lk, L.fresh = J.fresh;
  L.kfrom = 0, L.kto = -1;
  if (J.lq <= A.long_from) return L;
  L.mk = mask_args(A.mask, A.left, A.right, J.lq, J.lk);
  changing(A, J, L.mk, L.kfrom, L.kto);
  return L;
}

// 128 keys of a long segment and kv head, and this CTA's query tiles past them.
struct Item {
  Long s;
  int b, hk;
  int key0, key1;         // first and last key
  int qt0, n;             // first query tile with a row that sees one of them, number of this CTA's tiles
};
// What item_at and direct_at find of an item: its first key and this CTA's query tiles.
__device__ __forceinline__ void set_keys(const TcArgs& X, Item& I, int tile, int rank) {
  I.key0 = (I.s.kfrom / KM + tile) * KM;
  I.key1 = min(I.key0 + KM - 1, I.s.lk - 1);
  long long q_lo = 0, q_hi = I.s.lq - 1;
  if (I.s.mk.right >= 0) q_lo = max(q_lo, (long long)I.key0 - I.s.mk.off - I.s.mk.right);
  if (I.s.mk.left >= 0) q_hi = min(q_hi, (long long)I.key1 - I.s.mk.off + I.s.mk.left);
  I.qt0 = q_lo <= q_hi ? (int)(q_lo / X.tok) : 0;
  const int all = q_lo <= q_hi ? (int)(q_hi / X.tok) - I.qt0 + 1 : 0;
  I.n = all > rank ? (all - rank + X.share - 1) / X.share : 0;
}
// Item y of those listed: by segment, key tile, head.
__device__ __forceinline__ Item item_at(const TcArgs& X, const int* first, int c0, int y, int rank) {
  int lo = 0, hi = LIST;  // largest segment with first[lo] <= tile
  const int tile = y / X.a.c.hkv;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= tile) lo = mid;
    else hi = mid;
  }
  Item I;
  I.b = c0 + lo;
  I.hk = y - tile * X.a.c.hkv;
  I.s = long_at(X.a, I.b);
  set_keys(X, I, tile - first[lo], rank);
  return I;
}
// Place y of all that the bounds leave room for: by key tile, segment, head.  false: no item.
__device__ __forceinline__ bool direct_at(const TcArgs& X, int y, int rank, Item& I) {
  const int jobs = X.batch * X.a.c.hkv, tile = y / jobs, job = y - tile * jobs;
  I.b = job / X.a.c.hkv;
  I.hk = job - I.b * X.a.c.hkv;
  I.s = long_at(X.a, I.b);
  if (I.s.kfrom > I.s.kto || tile > I.s.kto / KM - I.s.kfrom / KM) return false;
  set_keys(X, I, tile, rank);
  return true;
}

// Where the weight and position of a key are.
__device__ __forceinline__ long long weight_at(const Args& A, const Item& I, int key, int page) {
  const int shift = A.c.page_shift;
  return (((long long)page * A.c.hkv + I.hk) << shift) + (key & ((1 << shift) - 1));
}
// The new weight of a key that got w, and a new key's position.
__device__ __forceinline__ void settle(const Args& A, const Item& I, int key, int page, float old, float w) {
  const long long at = weight_at(A, I, key, page);
  const bool fresh = key >= I.s.fresh;
  A.weight[at] = (fresh || A.decay == 0.f ? 0.f : A.decay * old) + w;
  if (fresh) A.position[at] = (int)((unsigned)key + (A.offsets ? (unsigned)__ldg(A.offsets + I.b) : 0u));
}

template <int DQK, typename T>
__global__ void __launch_bounds__(TC_THREADS, TcCfg<DQK>::RESIDENT) weigh_tc_kernel(const __grid_constant__ CUtensorMap q_map, const TcArgs X) {
  using C = TcCfg<DQK>;
  const Args& A = X.a;
  const int rank = blockIdx.x % X.share, me = blockIdx.x / X.share, step = gridDim.x / X.share;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // the swizzle counts from 1024
  float* s_nl = reinterpret_cast<float*>(smem + C::OFF_NL);
  int* s_tok = reinterpret_cast<int*>(smem + C::OFF_TOK);
  float* s_sum = reinterpret_cast<float*>(smem + C::OFF_SUM);
  int* s_odd = reinterpret_cast<int*>(smem + C::OFF_ODD);
  int* s_list = reinterpret_cast<int*>(smem + C::OFF_LIST);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* stop = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
  const TcCtx ctx{bar, stop}, own{bar, stop + 1};   // own: what this CTA has in flight, waited for in any case
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int used = X.tok * A.g;               // rows of a tile that are loaded
  const int shift = A.c.page_shift, in_page = (1 << shift) - 1;
  bool begun = false;                         // TMEM is held
  uint32_t tmem = 0;
  int passed = 0;                             // items of the lists before
  for (int c0 = 0; c0 < (X.places ? 1 : X.batch); c0 += LIST) {
    int items = X.places;
    if (!X.places) {
      // key tiles before each of up to LIST segments
      int tiles = 0;
      if (tid < LIST && c0 + tid < X.batch) {
        const Long L = long_at(A, c0 + tid);
        if (L.kfrom <= L.kto) tiles = L.kto / KM - L.kfrom / KM + 1;
      }
      int upto = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      if (lane == 31 && tid < LIST) s_list[LIST + 1 + warp] = upto;
      __syncthreads();
      int before = 0, total = 0;
#pragma unroll
      for (int w = 0; w < LIST / 32; ++w) {
        const int n = s_list[LIST + 1 + w];
        if (w < warp) before += n;
        total += n;
      }
      if (tid < LIST) s_list[tid] = before + upto - tiles;
      if (tid == 0) s_list[LIST] = total;
      __syncthreads();
      items = total * A.c.hkv;
    }
    // this CTA's: numbers me, me + step, ... of all lists
    int y = ((me - passed) % step + step) % step;
    passed += items;
    for (; y < items; y += step) {
      Item I;
      if (!X.places) I = item_at(X, s_list, c0, y, rank);
      else if (!direct_at(X, y, rank, I)) continue;
      const Long& J = I.s;
      const int n = I.n, key0 = I.key0, qt0 = I.qt0;
      if (tid == 0) {
        if (begun) {
          for (int i = 0; i < C::NBAR; ++i) mbar_inval(bar + i);
        }
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
        fence_mbar_init();
      }
      if (!begun) {
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
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      tmem = *tmem_holder;
      begun = true;

      auto load_tile = [&](int j) {           // query tile j of this CTA
        const int s = j % C::ST;
        mbar_arrive_expect_tx(bar + C::Q_FULL + s, C::NCH * 128 * used);
        const int row = J.q0 + (qt0 + rank + j * X.share) * X.tok;
        for (int c = 0; c < C::NCH; ++c)
          tma_load_3d(smem + C::OFF_Q + (s * C::NCH + c) * C::QCH, &q_map, bar + C::Q_FULL + s, c * 64, I.hk * A.g, row);
      };
      if (warp == LOAD_WARP && lane == 0)
        for (int j = 0; j < min(n, C::ST); ++j) load_tile(j);

      // the keys in 16 bits: 16 bytes become two swizzled pieces of 16; keys whose weights do
      // not change, and those of a page outside the cache, are zero
      const int* table = A.table + I.b * A.table_stride;
      auto page_of = [&](int key) {
        if (key < J.kfrom || key > J.kto) return -1;
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
            if (r < KM) {
              const int page = page_of(key0 + r);
              if (page >= 0)
                x[k] = __ldg(reinterpret_cast<const uint4*>(A.c.k + page * A.c.sk.p + ((key0 + r) & in_page) * A.c.sk.r +
                                                            I.hk * A.c.sk.h + c * 16));
            }
          }
#pragma unroll
          for (int k = 0; k < HELD; ++k) {
            const int i = i0 + k * TC_THREADS, r = i / PIECES, c = i - r * PIECES;
            if (r >= KM) continue;
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t v[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              v[2 * m] = widen2((uint16_t)w[m], (T*)nullptr);
              v[2 * m + 1] = widen2((uint16_t)(w[m] >> 16), (T*)nullptr);
            }
            uint8_t* at = smem + (c >> 2) * C::KCH + r * 128;
            const int p = (c & 3) * 2, sw = r & 7;
            *reinterpret_cast<uint4*>(at + ((p ^ sw) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(at + (((p + 1) ^ sw) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
          }
        }
        fence_proxy_async_smem();
      }
      __syncthreads();
      int page = -1;                          // exponentials: of this thread's key
      float old = 0.f;                        // and, of the first four warps, its weight before

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
          constexpr uint32_t ID = idesc_f16(KM, C::N, false, false, std::is_same<T, __half>::value);
          const uint64_t dk = sdesc_sw128(smem_u32(smem), 16, 1024);
          const uint64_t dq = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
          int j = 0;
          for (; j < n; ++j) {
            const int s = j % C::ST, sb = j & 1;
            if (!tc_wait(ctx, C::Q_FULL + s, (j / C::ST) & 1)) break;
            if (!tc_wait(ctx, C::S_EMPTY + sb, ((j >> 1) & 1) ^ 1)) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DQK / 16; ++ks) {
              const uint32_t off_k = (ks >> 2) * C::KCH + (ks & 3) * 32;
              const uint32_t off_q = (s * C::NCH + (ks >> 2)) * C::QCH + (ks & 3) * 32;
              umma_ss(tmem + sb * C::N, dk + (off_k >> 4), dq + (off_q >> 4), ID, ks > 0 ? 1u : 0u);
            }
            umma_commit(bar + C::S_FULL + sb);
            umma_commit(bar + C::Q_EMPTY + s);
          }
          // No product may be in flight when TMEM is released, and no commit may still signal a
          // barrier when the next item begins it anew.  Each signals its own, in no order that a
          // later one would tell of: all that nobody has to have waited for are waited for here.
          // (Rolled: unrolled, these loops spill 28 bytes of the other warps' registers, 2 us of 151.)
#pragma unroll 1
          for (int i = max(0, j - C::ST); i < j; ++i) tc_wait(own, C::Q_EMPTY + i % C::ST, (i / C::ST) & 1);
#pragma unroll 1
          for (int i = max(0, j - 2); i < j; ++i) tc_wait(own, C::S_FULL + (i & 1), (i >> 1) & 1);
        }
      } else if (warp == LSE_WARP) {
        // rows lane, lane + 32, ... of a tile; all loads of a tile are under way together,
        // a tile ahead of their use (each by itself, a trip to L2 apiece, they bound the kernel)
        int tok[C::N / 32];
        const float* head[C::N / 32];
#pragma unroll
        for (int k = 0; k < C::N / 32; ++k) {
          const int r = k * 32 + lane;
          tok[k] = s_tok[r];
          head[k] = A.lse + (long long)(I.hk * A.g + r - tok[k] * A.g) * A.total_q + J.q0;
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
        // --------------------------------------------------- exponentials
        const int half = warp >> 2, r = (warp & 3) * 32 + lane, key = key0 + r;
        constexpr int COLS = C::N / 2;
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * COLS;
        page = page_of(key);
        if (page < 0 && key >= J.kfrom && key <= J.kto) report(A, ATTN_ERR_BAD_PAGE);
        const float u = page >= 0 ? A.scale_log2 * exp2_int(kv_exp_of(__ldg(A.c.k_exp + (long long)page * A.c.hkv + I.hk))) : 0.f;
        if (page >= 0 && half == 0) old = A.weight[weight_at(A, I, key, page)];
        // tiles whose first token is at least need0 and whose last one is at most need1 see all keys
        const MaskArgs& mk = J.mk;
        const int need0 = mk.right >= 0 ? (int)max(0ll, (long long)I.key1 - mk.off - mk.right) : 0;
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
                const float2 a = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), u2, make_float2(l.x, l.y));
                const float2 b = fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), u2, make_float2(l.z, l.w));
                sum[0] = fma2(make_float2(fast_exp2(a.x), fast_exp2(a.y)), one2, sum[0]);
                sum[1] = fma2(make_float2(fast_exp2(b.x), fast_exp2(b.y)), one2, sum[1]);
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
      tc_fence_after();
      if (X.share > 1) cluster_sync();        // (the same items for all of a cluster)
      if (rank == 0 && tid < KM && page >= 0) {
        float w = s_sum[tid] + s_sum[KM + tid];
        for (int s = 1; s < X.share; ++s) w += peek(s_sum + tid, s) + peek(s_sum + KM + tid, s);
        settle(A, I, key0 + tid, page, old, w);
      }
      if (X.share > 1) cluster_sync();        // the sums have been read
    }
    __syncthreads();                          // the list has been used
  }
  if (begun && warp == MMA_WARP) {
    __syncwarp();
    tmem_dealloc(tmem, C::TMEM);
  }
  // Complete only after the short segments' kernel, beside which this one may run.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The bounded wait on a barrier that nobody completes, and again where another warp has
// given up before: out[0] = ATTN_ERR_TIMEOUT if the first ran out and said so, out[1] = 1
// if the second did not wait.
__global__ void __launch_bounds__(32) selftest_kernel(int* out) {
  constexpr uint64_t LIMIT = 1000000ull;   // 1 ms
  __shared__ __align__(8) uint64_t bar[1];
  __shared__ int stop[2];
  if (threadIdx.x != 0) return;
  stop[0] = 0, stop[1] = 1;
  mbar_init(bar, 1);
  fence_mbar_init();
  const TcCtx alone{bar, stop}, late{bar, stop + 1};
  const bool first = tc_wait<LIMIT>(alone, 0, 0);
  out[0] = !first && *alone.stop == 1 ? ATTN_ERR_TIMEOUT : ATTN_OK;
  const uint64_t t0 = globaltimer();
  const bool second = tc_wait<LIMIT>(late, 0, 0);
  out[1] = !second && globaltimer() - t0 < LIMIT / 2;
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
  x.batch = batch;
  x.tok = C::N / a.g;
  // most items: segments that q has room for, key tiles of max_k keys (one more where a
  // window begins inside a tile)
  const long long fit = a.total_q / (a.long_from + 1);
  const long long items = (fit < batch ? fit : batch) * a.c.hkv * (cdiv(a.max_k, KM) + 1LL);
  constexpr int CTAS = C::RESIDENT * SMS;
  x.share = 1;
  while (x.share < 8 && batch <= LIST && items * x.share * 2 <= CTAS) x.share *= 2;
  // a CTA per item, as a rule: the GPU deals them out as others end
  const long long places = (long long)batch * a.c.hkv * (cdiv(a.max_k, KM) + 1LL);
  x.places = x.share == 1 && places <= MAX_PLACES ? (int)places : 0;
  const int grid = x.places ? x.places : x.share > 1 ? (int)items * x.share : items < MAX_TC_GRID ? (int)items : MAX_TC_GRID;
  if (grid < 1) return ATTN_OK;
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
  cfg.gridDim = dim3(grid);
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

int launch_selftest(int* out, cudaStream_t st) {
  selftest_kernel<<<1, 32, 0, st>>>(out);
  return succeeded(cudaGetLastError()) ? ATTN_OK : ATTN_ERR_CUDA;
}

int long_group(int dqk) { return dqk <= 128 ? 128 : 64; }

int launch_long(const Args& a, bool bf16, int dqk, int batch, cudaStream_t st) {
  return bf16 ? launch_tc<__nv_bfloat16>(a, dqk, batch, st) : launch_tc<__half>(a, dqk, batch, st);
}

}  // namespace kvweigh
}  // namespace attn
