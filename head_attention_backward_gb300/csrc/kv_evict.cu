// Eviction from the paged cache by accumulated attention weight (attn_kv_evict).
//
// Per request and kv head the `keep` rows with the largest keys stay; a row's key is
// its weight, above all weights where its position is protected (where more than
// `keep` are protected, their weights, and 0 for all others).  Rows in front that
// go are holes, rows behind that stay fill them in order: every read is of a row
// >= keep and every write to a row < keep, so nothing has to wait for anything, and
// no more than min(keep, n - keep) rows move.
//
// * select_kernel: a cluster of 1 to 8 CTAs owns a request and head.  Its rows' keys
//   go to shared memory once (8 bytes a row read: weight and position); the least key
//   that stays is found digit by digit (11, 11 and 10 bits) from histograms that the
//   CTAs add up through each other's shared memory; two prefix sums over the rows
//   number the holes and those that fill them.  One more cluster checks the call and
//   counts the pages that go back.
// * move_kernel: a warp owns a page that has holes: the larger of its scale and of
//   those that come in, the rows that stay rounded again if it grew, then the rows.
//   One more CTA writes the lengths and the stack.
//
// Bound by memory where much goes (8 bytes a row, 2 (d_qk + d_v) a row that moves),
// by the dependent trips to memory and the barriers of the selection elsewhere.
#include "common.cuh"
#include "kv_common.cuh"

namespace attn {
namespace kvevict {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int HELD = 40 * 1024;         // keys of a CTA's share that fit shared memory
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_WARPS = MOVE_THREADS / 32;
constexpr uint32_t FIRST = 0xffffffffu; // key of a protected row

struct Args {
  attn_kv_evict_params p;
  KvCacheView c;
  int max_k;             // min(max_seqlen_k, max_blocks pages)
  int dqk, dv;
  int cluster;           // CTAs of a request and head
  int pages;             // of max_k tokens
  int half;              // most rows that move
  int spread;            // CTAs that share a request's and head's pages
  int* verdict;          // status of the call
  int4* plan;            // [batch]: length, length after, pages given back before it, unused
  int2* edge;            // [batch][kv head]: exponent bytes of the page that row `keep` is in
  int* holes;            // [batch][kv head][pages + 1]: holes before a page
  int* to;               // [batch][kv head][half]: rows of the holes, ascending
  int* from;             // and of what fills them, ascending
  uint32_t* keys;        // [batch][kv head][max_k], where they do not fit shared memory, else null
};

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((long long)tokens + (1 << shift) - 1) >> shift); }

// Whether a request shrinks, for lengths within their bounds.
__device__ __forceinline__ bool evicts(const Args& A, int n, int keep) {
  return n > 0 && n <= A.max_k && keep >= 0 && n > (long long)keep + A.p.slack;
}

// Keys order like weights; NaN is below every number, and above the 0 of a row that
// does not compete.  No weight's key is in the bin of FIRST.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 1;
  const uint32_t u = __float_as_uint(w + 0.f);       // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int rank_of() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
// The word at p of CTA `rank`'s shared memory.
__device__ __forceinline__ int peek(const void* p, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  int v;
  asm volatile("{\n\t.reg .u32 x;\n\tmapa.shared::cluster.u32 x, %1, %2;\n\tld.shared::cluster.u32 %0, [x];\n\t}"
               : "=r"(v) : "r"(a), "r"(rank) : "memory");
  return v;
}

__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Sum over the threads before this one; *total over all.  scratch: WARPS words, free
// for the next use after a barrier.
__device__ __forceinline__ int block_before(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = warp_scan(v);
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int x = scratch[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + s - v;
}

// The checks of the whole call, and where each request's pages go on the stack.
__device__ void check_call(const Args& A, int* scratch) {
  const attn_kv_evict_params& P = A.p;
  const int shift = A.c.page_shift, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int free_n = *P.free_count;
  bool bad = free_n < 0 || free_n > A.c.num_pages, off = false;
  long long given = 0;
  for (int b0 = 0; b0 < P.batch; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    int n = 0, after = 0, back = 0, total;
    if (b < P.batch) {
      const int keep = P.keep[b];
      n = after = P.seqlens[b];
      bad |= n < 0 || n > A.max_k || keep < -1;
      if (evicts(A, n, keep)) {
        after = keep;
        back = pages_of(n, shift) - pages_of(keep, shift);
      }
    }
    const int before = block_before(back, scratch, &total);
    if (b < P.batch) A.plan[b] = make_int4(n, after, (int)min(given + before, (long long)INT32_MAX), 0);
    given += total;
    __syncthreads();
  }
  bad |= given > A.c.num_pages - free_n;
  const bool any_bad = __syncthreads_or(bad);
  if (!any_bad) {
    for (int b = warp; b < P.batch; b += WARPS) {
      const int4 r = A.plan[b];
      if (r.x == r.y) continue;
      for (int i = lane; i < pages_of(r.x, shift); i += 32) {
        const int page = P.block_table[b * P.table_stride + i];
        off |= page < 0 || page >= A.c.num_pages;
      }
    }
  }
  const bool any_off = __syncthreads_or(off);
  if (threadIdx.x == 0) *A.verdict = any_bad ? ATTN_ERR_BAD_SEQLENS : any_off ? ATTN_ERR_BAD_PAGE : ATTN_OK;
}

__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ Args A) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int s_hist[BINS];
  __shared__ int s_scratch[2][WARPS];
  __shared__ int s_found[2], s_sum[3];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const attn_kv_evict_params& P = A.p;
  const int tid = threadIdx.x, rank = rank_of(), heads = A.c.hkv;
  const int job = blockIdx.x / A.cluster;
  if (job == P.batch * heads) {
    if (rank == 0) check_call(A, s_scratch[0]);
    return;
  }
  const int b = job / heads, h = job - b * heads;
  const int n = P.seqlens[b], keep = P.keep[b];
  if (!evicts(A, n, keep) || keep == 0) return;         // the same for the whole cluster
  const int shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int per = cdiv(n, A.cluster), lo = min(rank * per, n), mine = min(per, n - lo);
  uint32_t* keys = A.keys ? A.keys + (long long)job * A.max_k + lo : s_keys;
  const int* table = P.block_table + b * P.table_stride;
  const long long recent = (long long)n + P.position_offsets[b] - P.recent;
  auto fill = [&](bool protected_only) {
    for (int i = tid; i < mine; i += THREADS) {
      const int row = lo + i, page = table[row >> shift];
      uint32_t k = 0;
      if (page >= 0 && page < A.c.num_pages) {
        const long long at = (((long long)page * heads + h) << shift) + (row & in_page);
        const int pos = __ldg(P.weights.position + at);
        const uint32_t by_weight = key_of(__ldg(P.weights.weight + at));
        const bool first = pos < P.sink || pos >= recent;
        k = protected_only ? (first ? by_weight : 0) : first ? FIRST : by_weight;
      }
      keys[i] = k;
    }
  };
  fill(false);
  // the keep-th largest key
  uint32_t found = 0, mask = 0;
  int left = keep;                                       // rows to take among those that match so far
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int low = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < BINS; i += THREADS) s_hist[i] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < mine; i0 += THREADS) {
      const int i = i0 + tid;
      const uint32_t k = i < mine ? keys[i] : 0;
      const bool counts = i < mine && (k & mask) == found;
      const uint32_t digit = (k >> low) & ((1u << bits) - 1);
      const uint32_t who = __ballot_sync(0xffffffffu, counts);
      if (!who) continue;
      // a warp whose rows all fall into one bin (equal weights, protected rows) adds once
      const int leader = __ffs(who) - 1;
      const uint32_t one = __shfl_sync(0xffffffffu, digit, leader);
      if (__all_sync(0xffffffffu, !counts || digit == one)) {
        if ((tid & 31) == leader) atomicAdd(&s_hist[digit], __popc(who));
      } else if (counts) {
        atomicAdd(&s_hist[digit], 1);
      }
    }
    cluster_sync();
    // bins from the top: thread t has four, the last threads the lowest
    constexpr int PER = BINS / THREADS;
    int bin[PER], sum = 0, total;
    const int top = BINS - 1 - tid * PER;
#pragma unroll
    for (int j = 0; j < PER; ++j) bin[j] = 0;
    for (int r = 0; r < A.cluster; ++r) {
#pragma unroll
      for (int j = 0; j < PER; ++j) bin[j] += A.cluster == 1 ? s_hist[top - j] : peek(&s_hist[top - j], r);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += bin[j];
    int before = block_before(sum, s_scratch[pass & 1], &total);
    if (before < left && left <= before + sum) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (before < left && left <= before + bin[j]) {
          s_found[0] = top - j;
          s_found[1] = left - before;
        }
        before += bin[j];
      }
    }
    cluster_sync();                                      // also: the histograms have been read
    if (pass == 0 && s_found[0] == BINS - 1) {           // `keep` protected rows or more: among themselves
      fill(true);
      pass = -1;
      continue;
    }
    found |= (uint32_t)s_found[0] << low;
    left = s_found[1];
    mask |= ((1u << bits) - 1) << low;
  }
  // Rows of the least key: the first `left` of them stay.  A thread walks
  // neighbouring rows, an odd number of them so that the threads' lie in different banks.
  const int walk = cdiv(mine, THREADS) | 1, a = min(tid * walk, mine), z = min(a + walk, mine);
  int equal = 0, total;
  for (int i = a; i < z; ++i) equal += keys[i] == found;
  int ties = block_before(equal, s_scratch[1], &total);
  if (tid == 0) s_sum[0] = total;
  cluster_sync();
  for (int r = 0; r < rank; ++r) ties += peek(&s_sum[0], r);
  int holes = 0, fills = 0;
  {
    int t = ties;
    for (int i = a; i < z; ++i) {
      const uint32_t k = keys[i];
      const bool stays = k > found || (k == found && t < left);
      t += k == found;
      holes += lo + i < keep && !stays;
      fills += lo + i >= keep && stays;
    }
  }
  int total_holes, total_fills;
  const int holes0 = block_before(holes, s_scratch[0], &total_holes);
  __syncthreads();
  const int fills0 = block_before(fills, s_scratch[1], &total_fills);
  if (tid == 0) {
    s_sum[1] = total_holes;
    s_sum[2] = total_fills;
  }
  cluster_sync();
  holes = holes0;
  fills = fills0;
  for (int r = 0; r < rank; ++r) {
    holes += peek(&s_sum[1], r);
    fills += peek(&s_sum[2], r);
  }
  int* to = A.to + (long long)job * A.half;
  int* from = A.from + (long long)job * A.half;
  int* starts = A.holes + (long long)job * (A.pages + 1);
  for (int i = a; i < z; ++i) {
    const int row = lo + i;
    const uint32_t k = keys[i];
    const bool stays = k > found || (k == found && ties < left);
    ties += k == found;
    if (row < keep && (row & in_page) == 0) starts[row >> shift] = holes;
    if (row == keep) starts[pages_of(keep, shift)] = holes;
    if (row < keep && !stays) to[holes++] = row;
    if (row >= keep && stays) from[fills++] = row;
  }
  if (rank == 0 && tid == 0) {
    const int page = table[keep >> shift];
    if (page >= 0 && page < A.c.num_pages) {
      const long long at = (long long)page * heads + h;
      A.edge[job] = make_int2(A.c.k_exp[at], A.c.v_exp[at]);
    }
  }
  cluster_sync();                                        // no CTA leaves while others read its shared memory
}

// 16 e4m3 values times f, rounded again.
__device__ __forceinline__ uint4 times(const uint4& x, float f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = e4m3x2_to_h2((uint16_t)w[j]), hi = e4m3x2_to_h2((uint16_t)(w[j] >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    q[j] = f2_to_e4m3x2(a.x * f, a.y * f) | ((uint32_t)f2_to_e4m3x2(b.x * f, b.y * f) << 16);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

struct Side {
  uint8_t* x;            // of the head
  uint8_t* exp;
  long long page, row;   // strides
  int edge;              // exponent byte of the page that row `keep` is in, before the call
};

// The holes [h0, h1) of one page, on one side, by one warp.
template <int D>
__device__ __forceinline__ void fill_page(const Side& S, const int* table, const int* to, const int* from, int h0, int h1,
                                          int first, int rows, int edge_block, int shift, int heads) {
  constexpr int PER = D / 16;
  const int lane = threadIdx.x & 31, in_page = (1 << shift) - 1;
  const int page = table[first >> shift];
  uint8_t* exp_at = S.exp + (long long)page * heads;
  auto exp_of = [&](int row) {
    const int block = row >> shift;
    return kv_exp_of(block == edge_block ? (uint8_t)S.edge : S.exp[(long long)table[block] * heads]);
  };
  const int old = kv_exp_of(*exp_at);
  int e = old;
  for (int i = h0 + lane; i < h1; i += 32) e = max(e, exp_of(from[i]));
  e = __reduce_max_sync(0xffffffffu, e);
  uint8_t* dst = S.x + page * S.page;
  if (e > old) {
    // every row below `keep`, holes too: they are written after this
    const float f = exp2_int(old - e);
    for (int i = lane; i < rows * PER; i += 32) {
      uint4* at = reinterpret_cast<uint4*>(dst + (i / PER) * S.row + (i % PER) * 16);
      *at = times(*at, f);
    }
    if (lane == 0) *exp_at = (uint8_t)(e + KV_EXP_BIAS);
    __syncwarp();
  }
  constexpr int N = 4;   // pieces in flight
  const int all = (h1 - h0) * PER;
  for (int i0 = lane; i0 < all; i0 += 32 * N) {
    uint4 x[N];
    int ex[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + 32 * k;
      if (i < all) {
        const int row = from[h0 + i / PER];
        x[k] = *reinterpret_cast<const uint4*>(S.x + table[row >> shift] * S.page + (row & in_page) * S.row + (i % PER) * 16);
        ex[k] = exp_of(row);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + 32 * k;
      if (i < all)
        *reinterpret_cast<uint4*>(dst + (to[h0 + i / PER] & in_page) * S.row + (i % PER) * 16) =
            ex[k] == e ? x[k] : times(x[k], exp2_int(ex[k] - e));
    }
  }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const __grid_constant__ Args A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const attn_kv_evict_params& P = A.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int heads = A.c.hkv, verdict = *A.verdict;
  if (blockIdx.x == P.batch * heads * A.spread) {
    // lengths, offsets, the stack
    const int free_n = *P.free_count;
    __syncthreads();                                     // the output may be the same word
    int back = 0;
    for (int b = warp; b < P.batch; b += MOVE_WARPS) {
      const int4 r = A.plan[b];
      const bool goes = verdict == ATTN_OK && r.y < r.x;
      const int offset = P.position_offsets[b];
      const int need = pages_of(r.y, shift), held = pages_of(r.x, shift);
      __syncwarp();
      if (lane == 0) {
        P.seqlens_out[b] = goes ? r.y : r.x;
        P.position_offsets_out[b] = goes ? (int)((unsigned)offset + (unsigned)(r.x - r.y)) : offset;
      }
      if (!goes) continue;
      for (int i = lane; i < held - need; i += 32)
        P.free_pages[free_n + r.z + i] = P.block_table[b * P.table_stride + need + i];
      back = max(back, r.z + held - need);
    }
    __shared__ int s_back[MOVE_WARPS];
    if (lane == 0) s_back[warp] = back;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < MOVE_WARPS; ++w) back = max(back, s_back[w]);
      *P.free_count_out = free_n + back;
      *P.status = verdict;
    }
    return;
  }
  const int job = blockIdx.x / A.spread, share = blockIdx.x - job * A.spread;
  const int b = job / heads, h = job - b * heads;
  const int4 r = A.plan[b];
  if (verdict != ATTN_OK || r.y >= r.x) return;
  const int keep = r.y, pages = pages_of(keep, shift);
  const int* table = P.block_table + b * P.table_stride;
  const int* to = A.to + (long long)job * A.half;
  const int* from = A.from + (long long)job * A.half;
  const int* starts = A.holes + (long long)job * (A.pages + 1);
  const int2 edge = A.edge[job];
  const Side K{A.c.k + h * A.c.sk.h, A.c.k_exp + h, A.c.sk.p, A.c.sk.r, edge.x};
  const Side V{A.c.v + h * A.c.sv.h, A.c.v_exp + h, A.c.sv.p, A.c.sv.r, edge.y};
  for (int p = share * MOVE_WARPS + warp; p < pages; p += A.spread * MOVE_WARPS) {
    const int h0 = starts[p], h1 = starts[p + 1], first = p << shift, rows = min(1 << shift, keep - first);
    if (h0 == h1) continue;
    fill_page<DQK>(K, table, to, from, h0, h1, first, rows, keep >> shift, shift, heads);
    fill_page<DV>(V, table, to, from, h0, h1, first, rows, keep >> shift, shift, heads);
    const long long own = ((long long)table[p] * heads + h) << shift;
    for (int i = h0 + lane; i < h1; i += 32) {
      const int row = from[i];
      const long long src = (((long long)table[row >> shift] * heads + h) << shift) + (row & in_page);
      const long long dst = own + (to[i] & in_page);
      P.weights.weight[dst] = P.weights.weight[src];
      P.weights.position[dst] = P.weights.position[src];
    }
  }
}

struct Layout {
  size_t off_plan, off_edge, off_holes, off_to, off_from, off_keys, total;
  int cluster, pages, half, max_k;
  bool held;
};

static int layout(const attn_kv_evict_params* p, Layout* L) {
  if (!p || p->reserved != 0) return ATTN_ERR_INVALID_ARG;
  const attn_kv_cache& c = p->cache;
  const int shift = kv_page_shift(c.page_size);
  if (shift < 0 || c.num_pages < 1 || c.nhead_kv < 1 || c.nhead_kv > KV_MAX_HEADS) return ATTN_ERR_INVALID_ARG;
  if (p->batch < 1 || p->batch > ATTN_KV_MAX_BATCH || p->max_seqlen_k < 0 || p->max_blocks < 1 ||
      ((long long)p->max_blocks << shift) > (1LL << 30) || p->table_stride < p->max_blocks || p->table_stride >= (1LL << 36))
    return ATTN_ERR_INVALID_ARG;
  if (p->sink < 0 || p->recent < 0 || p->slack < 0 || (long long)p->batch * c.nhead_kv > (1 << 24)) return ATTN_ERR_INVALID_ARG;
  const long long cap = (long long)p->max_blocks << shift;
  L->max_k = p->max_seqlen_k < cap ? p->max_seqlen_k : (int)cap;
  // Rows of a CTA: enough for its threads, few enough for its shared memory.
  L->cluster = 1;
  while (L->cluster < 8 && cdiv(L->max_k, L->cluster) > 8192) L->cluster *= 2;
  L->held = cdiv(L->max_k, L->cluster) <= HELD;
  L->pages = cdiv(L->max_k, c.page_size);
  L->half = L->max_k / 2 + 1;
  const size_t jobs = (size_t)p->batch * c.nhead_kv;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  size_t o = 256;
  L->off_plan = o;  o = up(o + (size_t)p->batch * sizeof(int4));
  L->off_edge = o;  o = up(o + jobs * sizeof(int2));
  L->off_holes = o; o = up(o + jobs * (L->pages + 1) * sizeof(int));
  L->off_to = o;    o = up(o + jobs * L->half * sizeof(int));
  L->off_from = o;  o = up(o + jobs * L->half * sizeof(int));
  L->off_keys = o;  o = up(o + (L->held ? 0 : jobs * L->max_k * sizeof(uint32_t)));
  L->total = o;
  return ATTN_OK;
}

template <int DQK, int DV>
static cudaError_t launch_move(const cudaLaunchConfig_t& cfg, const Args& a) {
  return cudaLaunchKernelEx(&cfg, move_kernel<DQK, DV>, a);
}

static int run(const attn_kv_evict_params* p, void* ws, size_t bytes, cudaStream_t st) {
  Layout L;
  int s = layout(p, &L);
  if (s != ATTN_OK) return s;
  Args a{};
  if ((s = kv_resolve(p->cache, &a.c)) != ATTN_OK) return s;
  const void* need[] = {p->keep, p->seqlens, p->seqlens_out, p->position_offsets, p->position_offsets_out, p->block_table,
                        p->free_pages, p->free_count, p->free_count_out, p->status, p->weights.weight, p->weights.position};
  for (const void* x : need)
    if (!x || !aligned_to(x, 4)) return ATTN_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256)) return ATTN_ERR_INVALID_ARG;
  if (bytes < L.total) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  char* w = static_cast<char*>(ws);
  a.p = *p;
  a.max_k = L.max_k;
  a.dqk = p->cache.d_qk;
  a.dv = p->cache.d_v;
  a.cluster = L.cluster;
  a.pages = L.pages;
  a.half = L.half;
  a.verdict = reinterpret_cast<int*>(w);
  a.plan = reinterpret_cast<int4*>(w + L.off_plan);
  a.edge = reinterpret_cast<int2*>(w + L.off_edge);
  a.holes = reinterpret_cast<int*>(w + L.off_holes);
  a.to = reinterpret_cast<int*>(w + L.off_to);
  a.from = reinterpret_cast<int*>(w + L.off_from);
  a.keys = L.held ? nullptr : reinterpret_cast<uint32_t*>(w + L.off_keys);
  const int jobs = p->batch * p->cache.nhead_kv;
  const int share = 8 * SMS / jobs, whole = cdiv(L.pages, MOVE_WARPS);
  a.spread = share < 1 || whole < 1 ? 1 : share < whole ? share : whole;
  const size_t smem = L.held ? (size_t)cdiv(L.max_k, L.cluster) * sizeof(uint32_t) : 0;
  if (smem > 32 * 1024 && !succeeded(cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                          (int)(HELD * sizeof(uint32_t)))))
    return ATTN_ERR_CUDA;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = L.cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((jobs + 1) * L.cluster);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (!succeeded(cudaLaunchKernelEx(&cfg, select_kernel, a))) return ATTN_ERR_CUDA;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(jobs * a.spread + 1);
  cfg.blockDim = dim3(MOVE_THREADS);
  cfg.dynamicSmemBytes = 0;
  const cudaError_t e = a.dqk == 64    ? launch_move<64, 64>(cfg, a)
                        : a.dqk == 128 ? launch_move<128, 128>(cfg, a)
                        : a.dqk == 192 ? launch_move<192, 128>(cfg, a)
                                       : launch_move<256, 256>(cfg, a);
  return succeeded(e) ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace kvevict
}  // namespace attn

extern "C" int attn_kv_evict_workspace_size(const attn_kv_evict_params* p, size_t* bytes) {
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  *bytes = 0;
  attn::kvevict::Layout L;
  const int s = attn::kvevict::layout(p, &L);
  if (s == ATTN_OK) *bytes = L.total;
  return s;
}

extern "C" int attn_kv_evict(const attn_kv_evict_params* p, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return attn::kvevict::run(p, workspace, workspace_bytes, stream);
}
