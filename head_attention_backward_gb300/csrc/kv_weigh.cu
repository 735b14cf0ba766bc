// Attention weights of cached tokens (attn_kv_weigh):
//
//   w[page, head, row] <- decay w + sum over query rows and heads of the group of
//                         exp(s q k - LSE),   K = 2^ek Kq per page and kv head.
//
// The softmax is not computed again: the LSE of the attention call is its
// normaliser, so one pass over K is enough, V is not read, and every key's sum is
// its own: no maximum, no rescaling, nothing to join between CTAs and no atomics.
// Decoding is bound by memory (1 byte a K value, a quarter of attention's flops a
// byte), long segments by the products and the exponentials: kv_weigh_tc.cu.
//
// * A CTA owns one request, kv head and split of the keys.  The query rows (token x
//   head of the group) lie in shared memory as fp16 fragments under a power-of-two
//   scale per row, which is exact unless an element is 2^-28 of its row's largest.
// * A warp takes tiles of 16 keys in turn, through a ring of its own in shared memory
//   that each lane fills for itself with asynchronous copies.  S^T = K Q^T in
//   m16n8k16 products: the 16-row side holds the keys, so a key's sum over query rows
//   is in four lanes of one warp.  The contraction's order is free, so a lane takes
//   16 consecutive bytes of a K row as its share of four k-steps: one wide load,
//   e4m3 to fp16 in one conversion per two values, exactly.
// * Scores, exponentials, sums and weights are fp32.
#include <cmath>

#include "kv_weigh.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace kvweigh {

constexpr int TILE = 16;
constexpr int CHUNK = 128;          // query rows in shared memory at a time
// Query rows (tokens x heads of the group) of a segment beyond which it goes to the
// tensor cores.  8 requests of 4,000 tokens, 8 kv heads of 128: 128 rows 38 us here,
// 47 us there; 256 rows 74 and 55.  4 requests, 4 heads of 192: 96 rows 21 and 21, 128
// rows 25 and 19; of 256: 27 and 29, 32 and 28.
constexpr int LONG_ROWS = 128;

template <typename T> __device__ __forceinline__ float2 up2(uint32_t x);
template <> __device__ __forceinline__ float2 up2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 up2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Copies of a lane's own, read back by that lane alone: no barrier joins the lanes.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// ONE: at most eight query rows, whose fragments stay in registers.
template <int DQK, bool ONE>
struct Cfg {
  // More, smaller CTAs where their shared memory is the rings alone: one's beginning hides
  // under more others (64 requests of up to 8,192 tokens, 8 heads of 128: 62 us; 65 with 8
  // warps, three CTAs per SM and a tile more in each ring; 63 with 2 warps).
  static constexpr int NWARPS = ONE ? 4 : 8;
  static constexpr int MIN_TILES = 2 * NWARPS;   // of a split
  // More CTAs than reside even out ragged requests, as long as a warp's share stays FULL_TILES
  // / NWARPS tiles: MAX_GRID of them at most (the same call: 62 us, 64 with 2,128, 71 with
  // one wave; 16 requests of up to 2,000: 9.4 with all of MIN_TILES, one wave 7.9).
  static constexpr int FULL_TILES = ONE ? 8 * NWARPS : MIN_TILES;
  static constexpr int MAX_GRID = ONE ? 3600 : 1536;
  static constexpr int PIECES = DQK / 64;    // 16-byte pieces of a K row in a lane
  static constexpr int FRAGS = DQK / 32;     // 16-byte pieces of a row group's fragments in a lane
  static constexpr int RESIDENT = ONE ? (DQK <= 128 ? 7 : 4) : DQK <= 128 ? 3 : 2;
  static constexpr int DEPTH = DQK == 64 ? (ONE ? 5 : 6) : DQK == 256 ? 3 : ONE && DQK == 128 ? 3 : 4;   // tiles of a warp's ring
  static constexpr int STAGE = TILE * DQK + 128;                     // and 16 old weights
  static constexpr int RING = NWARPS * DEPTH * STAGE;
  static constexpr int GROUP = FRAGS * 32 * 16;                      // a row group's fragments
};

template <int DQK, typename T, bool ONE>
__global__ void __launch_bounds__(32 * Cfg<DQK, ONE>::NWARPS, Cfg<DQK, ONE>::RESIDENT) weigh_kernel(const Args A) {
  using C = Cfg<DQK, ONE>;
  constexpr int NWARPS = C::NWARPS;
  constexpr int PIECES = C::PIECES, FRAGS = C::FRAGS, DEPTH = C::DEPTH;
  extern __shared__ uint4 s_all[];           // the warps' rings, then the fragments: [row group][FRAGS][lane]
  uint4* s_q = s_all + C::RING / 16;
  __shared__ float2 s_row[CHUNK];            // log2 units per raw score, negated log2-scaled LSE
  __shared__ int s_tok[CHUNK];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the long segments' kernel
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int job = blockIdx.x / A.nsplit, split = blockIdx.x - job * A.nsplit;
  const int b = job / A.c.hkv, hk = job - b * A.c.hkv;
  const Segment J = segment_of(A, b);
  if (J.bad && tid == 0 && split == 0 && hk == 0) report(A, ATTN_ERR_BAD_SEQLENS);
  if (J.lq <= 0 || J.lq > A.long_from) return;
  const MaskArgs mk = mask_args(A.mask, A.left, A.right, J.lq, J.lk);
  int kfrom, kto;
  changing(A, J, mk, kfrom, kto);
  const int k0 = kfrom & ~(TILE - 1), ntile_all = kto >= kfrom ? (kto - k0) / TILE + 1 : 0;
  const int per = cdiv(max(C::MIN_TILES, cdiv(ntile_all, A.nsplit)), NWARPS) * NWARPS;
  const int tile0 = split * per, ntile = min(per, ntile_all - tile0);
  if (ntile <= 0) return;
  const int key0 = k0 + (tile0 + warp) * TILE;              // this warp's first tile, then every NWARPS-th
  constexpr int STEP = NWARPS * TILE;
  const int mine = cdiv(ntile - warp, NWARPS);
  const int shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int* table = A.table + b * A.table_stride;
  const int offset = A.offsets ? __ldg(A.offsets + b) : 0;
  const uint8_t* kbase = A.c.k + hk * A.c.sk.h + (long long)g * A.c.sk.r + t * 16;
  const long long krow8 = 8 * A.c.sk.r;
  const int own = g + 8 * t;                                // the key of a tile that lane t < 2 writes
  const uint32_t ring = ptx::smem_u32(s_all) + warp * DEPTH * C::STAGE + lane * 16;
  const uint32_t wring = ptx::smem_u32(s_all) + warp * DEPTH * C::STAGE + TILE * DQK + lane * 4;
  const int nrow = J.lq * A.g;

  for (int r0 = 0; r0 < nrow; r0 += CHUNK) {
    const int rows = min(CHUNK, nrow - r0), groups = ONE ? 1 : cdiv(rows, 8);
    const int i0 = r0 / A.g, i1 = (r0 + rows - 1) / A.g;
    const bool first = r0 == 0;
    int vlo, vhi;                            // keys that any row of the chunk sees
    seen_by(mk, J.lk, i0, i1, vlo, vhi);
    // keys that all of them see (keys past the last one are never written)
    const int flo = mk.left >= 0 ? (int)max(0ll, (long long)i1 + mk.off - mk.left) : 0;
    const int fhi = mk.right >= 0 ? (int)max(-1ll, min((long long)INT32_MAX, (long long)i0 + mk.off + mk.right)) : INT32_MAX;
    bool staged = false, odd = false;        // odd: a row of the chunk adds nothing, not even NaN
    float2 row[2];
    uint4 qf[ONE ? FRAGS : 1];

    for (int base = 0; base < mine || !staged; base += 32) {
      // This warp's next 32 tiles, a lane each: addresses, scale, and what the others ask
      // of them as bits.  Worked out per tile by all lanes, they were half of the
      // instructions, which bound the kernel.
      const int count = min(32, mine - base), key_base = key0 + base * STEP;
      long long k_at = 0, w_at = 0;
      float scale = 0.f;
      uint32_t has, views, wholes;           // tiles with a page; that a row sees; that all rows see
      {
        const int key = key_base + lane * STEP;
        bool ok = false;
        if (lane < count) {
          const int page = __ldg(table + (key >> shift));
          ok = page >= 0 && page < A.c.num_pages;
          if (ok) {
            const long long at = (long long)page * A.c.hkv + hk;
            scale = exp2_int(kv_exp_of(__ldg(A.c.k_exp + at)));
            k_at = page * A.c.sk.p + (long long)(key & in_page) * A.c.sk.r;
            w_at = (at << shift) + (key & in_page);
          } else {
            report(A, ATTN_ERR_BAD_PAGE);
          }
        }
        has = __ballot_sync(0xffffffffu, ok);
        views = __ballot_sync(0xffffffffu, ok && key <= vhi && key + TILE - 1 >= vlo);
        wholes = __ballot_sync(0xffffffffu, key >= flo && key + TILE - 1 <= fhi);
      }
      // tile j into its stage; a group per tile, empty ones too
      auto load = [&](int j, int stage) {
        if (j < count) {
          const long long ka = __shfl_sync(0xffffffffu, k_at, j), wa = __shfl_sync(0xffffffffu, w_at, j);
          if (views >> j & 1) {
            const uint8_t* p = kbase + ka;
            const uint8_t* p8 = p + krow8;
            const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
            for (int c = 0; c < PIECES; ++c) {
              cp16(dst + c * 1024, p + c * 64);
              cp16(dst + c * 1024 + 512, p8 + c * 64);
            }
          }
          if (t < 2 && first && (has >> j & 1)) cp4(wring + stage * C::STAGE, A.weight + wa + own);
        }
        cp_commit();
      };
#pragma unroll
      for (int j = 0; j < DEPTH - 1; ++j) load(j, j);

      if (!staged) {
        // rows of this chunk, a row group per warp: row g's share of lane t are the 16
        // elements at pieces t + 4 c; rows that add nothing are zero
        if (!first) __syncthreads();
        bool without = false;
        for (int n = warp; n < groups; n += NWARPS) {
          const int rr = 8 * n + g;
          const int rl = r0 + min(rr, rows - 1);
          const int i = rl / A.g;
          const int h = hk * A.g + rl - i * A.g;
          const T* qp = static_cast<const T*>(A.q) + elem_off(A.sq, (long long)J.q0 + i, h);
          const float l = __ldg(A.lse + (long long)h * A.total_q + J.q0 + i);
          const bool adds = rr < rows && fabsf(l) < INFINITY;
          without |= rr < rows && !adds;
          uint4 raw[FRAGS];
          float mx = 0.f;
#pragma unroll
          for (int c = 0; c < PIECES; ++c) {
            const uint4* p = reinterpret_cast<const uint4*>(qp + (t + 4 * c) * 16);
            raw[2 * c] = __ldg(p);
            raw[2 * c + 1] = __ldg(p + 1);
          }
#pragma unroll
          for (int x = 0; x < FRAGS; ++x) {
            if (!adds) raw[x] = make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = up2<T>(w[k]);
              mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          int e = (int)(__float_as_uint(mx) >> 23) - 127;
          e = e == 128 ? 14 : max(e, -100);      // infinities stay what they are
          const float up = exp2_int(14 - e);
#pragma unroll
          for (int x = 0; x < FRAGS; ++x) {
            const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = up2<T>(w[k]);
              y[k] = pack_h2(f.x * up, f.y * up);
            }
            s_q[(n * FRAGS + x) * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);
          }
          if (t == 0) {
            s_row[rr] = make_float2(A.scale_log2 * exp2_int(e - 14), adds ? -l * 1.4426950408889634f : -INFINITY);
            s_tok[rr] = i;
          }
        }
        odd = __syncthreads_or(without);
        staged = true;
        if (ONE) {
#pragma unroll
          for (int x = 0; x < FRAGS; ++x) qf[ONE ? x : 0] = s_q[x * 32 + lane];
          row[0] = s_row[2 * t];
          row[1] = s_row[2 * t + 1];
        }
      }

      if (odd) wholes = 0;
      for (int j0 = 0; j0 < count; j0 += DEPTH) {
#pragma unroll
      for (int stage = 0; stage < DEPTH; ++stage) {      // tile j is in stage j % DEPTH
        const int j = j0 + stage;
        if (j >= count) break;
        load(j + DEPTH - 1, (stage + DEPTH - 1) % DEPTH);
        cp_wait<DEPTH - 1>();
        const int key = key_base + j * STEP;
        const float u = __shfl_sync(0xffffffffu, scale, j);
        const long long wa = __shfl_sync(0xffffffffu, w_at, j);
        const uint32_t src = ring + stage * C::STAGE, old_at = wring + stage * C::STAGE;
        const bool in_view = views >> j & 1;
        if (!(has >> j & 1) || (!first && !in_view)) continue;
        float sum[2] = {0.f, 0.f};
        if (in_view) {
          uint4 k[PIECES][2];
#pragma unroll
          for (int c = 0; c < PIECES; ++c) {
            k[c][0] = lds128(src + c * 1024);
            k[c][1] = lds128(src + c * 1024 + 512);
          }
          for (int n = 0; n < groups; ++n) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < FRAGS; ++x) {
              const uint4 q = ONE ? qf[ONE ? x : 0] : s_q[(n * FRAGS + x) * 32 + lane];
              const uint4 &ra = k[x >> 1][0], &rb = k[x >> 1][1];
              const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const int word = (x & 1) * 2 + s;
                const uint32_t a[4] = {e4m3x2_to_h2((uint16_t)wa[word]), e4m3x2_to_h2((uint16_t)wb[word]),
                                       e4m3x2_to_h2((uint16_t)(wa[word] >> 16)), e4m3x2_to_h2((uint16_t)(wb[word] >> 16))};
                mma16816(acc, a, s ? q.z : q.x, s ? q.w : q.y);
              }
            }
            if (!ONE) {
              row[0] = s_row[8 * n + 2 * t];
              row[1] = s_row[8 * n + 2 * t + 1];
            }
            float p[2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) p[r][kk] = fast_exp2(fmaf(acc[2 * kk + r], row[r].x * u, row[r].y));
            if (!(wholes >> j & 1)) {
#pragma unroll
              for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                  if (row[r].y == -INFINITY || !sees(mk, s_tok[8 * n + 2 * t + r], key + g + 8 * kk)) p[r][kk] = 0.f;
            }
            sum[0] += p[0][0] + p[1][0];
            sum[1] += p[0][1] + p[1][1];
          }
          // over the four lanes; even lanes end with key g, odd ones with key g + 8
          const bool right = t & 1;
          const float other = __shfl_xor_sync(0xffffffffu, right ? sum[0] : sum[1], 1);
          sum[0] = (right ? sum[1] : sum[0]) + other;
          sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
        }
        const int at_key = key + own;
        if (t < 2 && at_key >= kfrom && at_key <= kto) {
          float* w = A.weight + wa + own;
          // (a later chunk adds to what this lane wrote before)
          float old = first ? lds32(old_at) * A.decay : *w;
          const bool is_fresh = at_key >= J.fresh;
          if (first && (is_fresh || A.decay == 0.f)) old = 0.f;
          *w = old + sum[0];
          if (first && is_fresh) A.position[wa + own] = (int)((unsigned)at_key + (unsigned)offset);
        }
      }
      }
      cp_wait<0>();
    }
  }
}

template <int DQK, typename T, bool ONE>
static int launch_rows(Args a, int jobs, int groups, cudaStream_t st) {
  using C = Cfg<DQK, ONE>;
  const int tiles = cdiv(a.max_k, TILE), wave = C::RESIDENT * SMS / jobs, many = C::MAX_GRID / jobs;
  const int full = cdiv(tiles, C::FULL_TILES), least = cdiv(tiles, C::MIN_TILES);
  a.nsplit = full < many ? full : many;
  if (a.nsplit < wave) a.nsplit = wave < least ? wave : least;
  if (a.nsplit < 1) a.nsplit = 1;
  // the limit is the kernel's, always the same one
  constexpr int MOST = C::RING + (ONE ? 1 : CHUNK / 8) * C::GROUP;
  if (!succeeded(cudaFuncSetAttribute(weigh_kernel<DQK, T, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST)))
    return ATTN_ERR_CUDA;
  weigh_kernel<DQK, T, ONE><<<jobs * a.nsplit, 32 * C::NWARPS, C::RING + groups * C::GROUP, st>>>(a);
  return succeeded(cudaGetLastError()) ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int DQK, typename T>
static int launch(const Args& a, int jobs, int groups, cudaStream_t st) {
  return groups <= 1 ? launch_rows<DQK, T, true>(a, jobs, 1, st) : launch_rows<DQK, T, false>(a, jobs, groups, st);
}

template <typename T>
static int launch(const Args& a, int dqk, int jobs, int groups, cudaStream_t st) {
  if (dqk == 64) return launch<64, T>(a, jobs, groups, st);
  if (dqk == 128) return launch<128, T>(a, jobs, groups, st);
  if (dqk == 192) return launch<192, T>(a, jobs, groups, st);
  return launch<256, T>(a, jobs, groups, st);
}

static int run(const attn_kv_weigh_params* p, cudaStream_t st) {
  if (!p || (p->dtype != ATTN_BF16 && p->dtype != ATTN_FP16)) return ATTN_ERR_INVALID_ARG;
  Args a{};
  const int s = kv_resolve(p->cache, &a.c);
  if (s != ATTN_OK) return s;
  if (p->batch < 1 || p->nhead_q < 1 || p->nhead_q % p->cache.nhead_kv != 0 || p->total_q < 0 || p->max_seqlen_q < 0 ||
      p->max_seqlen_k < 0 || p->max_blocks < 1 || p->table_stride < p->max_blocks || p->table_stride >= (1LL << 36))
    return ATTN_ERR_INVALID_ARG;
  if (p->total_q > (1 << 30) || ((long long)p->max_blocks << a.c.page_shift) > (1LL << 30) ||
      (long long)p->batch * p->cache.nhead_kv > (1 << 24) || p->nhead_q > (1 << 20))
    return ATTN_ERR_INVALID_ARG;
  if (p->mask < ATTN_MASK_NONE || p->mask > ATTN_MASK_WINDOW) return ATTN_ERR_INVALID_ARG;
  if (p->mask == ATTN_MASK_WINDOW && (p->window_left < -1 || p->window_right < -1)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->softmax_scale) || p->softmax_scale == 0.f || !std::isfinite(p->decay) || p->decay < 0.f)
    return ATTN_ERR_INVALID_ARG;
  const void* words[] = {p->cu_seqlens_q, p->seqlens_k, p->block_table, p->weights.weight, p->weights.position, p->weights.status};
  for (const void* x : words)
    if (!x || !aligned_to(x, 4)) return ATTN_ERR_INVALID_ARG;
  if (!aligned_to(p->cu_seqlens_q_padded, 4) || !aligned_to(p->position_offsets, 4) || !aligned_to(p->new_lens, 4) || !aligned_to(p->lse, 4) ||
      !aligned_to(p->q, 16) || !packed_strides(p->stride_q, p->nhead_q, p->cache.d_qk, &a.sq))
    return ATTN_ERR_INVALID_ARG;
  if (p->total_q == 0) return ATTN_OK;
  if (!p->q || !p->lse) return ATTN_ERR_INVALID_ARG;
  a.q = p->q;
  a.lse = p->lse;
  a.cu_q = p->cu_seqlens_q;
  a.st_q = p->cu_seqlens_q_padded ? p->cu_seqlens_q_padded : p->cu_seqlens_q;
  a.len_k = p->seqlens_k;
  a.table = p->block_table;
  a.table_stride = p->table_stride;
  a.offsets = p->position_offsets;
  a.new_lens = p->new_lens;
  const long long cap = (long long)p->max_blocks << a.c.page_shift;
  a.max_k = p->max_seqlen_k < cap ? p->max_seqlen_k : (int)cap;
  a.total_q = p->total_q;
  a.max_q = p->max_seqlen_q;
  a.hq = p->nhead_q;
  a.g = p->nhead_q / p->cache.nhead_kv;
  a.mask = p->mask;
  a.left = p->mask == ATTN_MASK_WINDOW ? p->window_left : -1;
  a.right = p->mask == ATTN_MASK_WINDOW ? p->window_right : -1;
  a.fresh = p->mask == ATTN_MASK_CAUSAL_BOTTOM_RIGHT || p->mask == ATTN_MASK_WINDOW;
  a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  a.decay = p->decay;
  a.weight = p->weights.weight;
  a.position = p->weights.position;
  a.status = p->weights.status;
  // Segments of more query rows than LONG_ROWS go to the tensor cores.
  a.long_from = a.g <= long_group(p->cache.d_qk) ? LONG_ROWS / a.g : 1 << 30;
  const int jobs = p->batch * p->cache.nhead_kv;
  const long long most = (long long)(p->max_seqlen_q < p->total_q ? p->max_seqlen_q : p->total_q) * a.g;
  const int groups = cdiv(most < CHUNK ? (int)most : CHUNK, 8);
  const bool bf16 = p->dtype == ATTN_BF16;
  const int s2 = bf16 ? launch<__nv_bfloat16>(a, p->cache.d_qk, jobs, groups, st)
                      : launch<__half>(a, p->cache.d_qk, jobs, groups, st);
  if (s2 != ATTN_OK || most <= (long long)a.long_from * a.g) return s2;
  return launch_long(a, bf16, p->cache.d_qk, p->batch, st);
}

}  // namespace kvweigh
}  // namespace attn

extern "C" int attn_kv_weigh(const attn_kv_weigh_params* p, cudaStream_t stream) { return attn::kvweigh::run(p, stream); }
