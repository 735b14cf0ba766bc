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
//   go to shared memory once (8 bytes a row read: weight and position), several rows of
//   a thread on their way together; the least key that stays is found digit by digit
//   (11, 11 and 10 bits) from histograms that the CTAs add up through each other's
//   shared memory; two prefix sums over the rows number the holes and those that fill
//   them.  A few more CTAs check the call and count the pages that go back.
// * move_kernel: a CTA owns a stretch of a request's and head's pages: the larger of a
//   page's scale and of those that come in, the rows that stay rounded again where it
//   grew, then the rows.  One more CTA writes the lengths and the stack.
//
// Bound by memory where much goes (8 bytes a row, 2 (d_qk + d_v) a row that moves),
// by the dependent trips to memory and the barriers of the selection elsewhere.
#include "common.cuh"
#include "kv_common.cuh"

namespace attn {
namespace kvevict {

// Threads of a CTA of select_kernel: two CTAs per SM where one owns a request and head,
// more threads per row where several do (131,072 rows, 8 heads: 35 us, 38 with 512).
constexpr int ONE_THREADS = 512, MANY_THREADS = 1024;
constexpr int MAX_WARPS = MANY_THREADS / 32;
constexpr int BINS = 2048;
constexpr int HELD = 40 * 1024;         // keys of a CTA's share that fit shared memory
// Clusters of 16 are no help: their CTAs need 16 SMs of a GPC at a time, and eight heads'
// clusters ran in two turns (131,072 rows: 61 us against 38 with eight CTAs).
constexpr int MAX_CLUSTER = 8;
constexpr int SHARE = 8192;             // rows of a CTA that its cluster grows for
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_WARPS = MOVE_THREADS / 32;
constexpr int CHUNK = 1024;             // rows that a CTA of move_kernel works on at a time
constexpr int CHUNK_PAGES = CHUNK / 16;
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
  int checks;            // CTAs that check the call, at most MOVE_THREADS
  int* verdict;          // status of the call, but for its pages
  int* off;              // [checks]: pages outside the cache
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

// A barrier of the CTAs that own a request and head (a cluster's costs a microsecond).
template <bool ONE>
__device__ __forceinline__ void owners_sync() {
  if (ONE) __syncthreads();
  else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

__device__ __forceinline__ int4 peek4(const void* p, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  int4 v;
  asm volatile("{\n\t.reg .u32 x;\n\tmapa.shared::cluster.u32 x, %4, %5;\n\tld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [x];\n\t}"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "r"(rank) : "memory");
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

// Sum over the threads before this one; *total over all.  scratch: MAX_WARPS words, free
// for the next use after a barrier.
template <int THREADS>
__device__ __forceinline__ int block_before(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = warp_scan(v);
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int x = scratch[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + s - v;
}

// The checks of the whole call by A.checks CTAs, and (the first of them) where each
// request's pages go on the stack.
template <int THREADS>
__device__ void check_call(const Args& A, int part, int* scratch) {
  constexpr int WARPS = THREADS / 32;
  const attn_kv_evict_params& P = A.p;
  const int shift = A.c.page_shift, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (part == 0) {
    const int free_n = *P.free_count;
    bool bad = free_n < 0 || free_n > A.c.num_pages;
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
      const int before = block_before<THREADS>(back, scratch, &total);
      if (b < P.batch) A.plan[b] = make_int4(n, after, (int)min(given + before, (long long)INT32_MAX), 0);
      given += total;
      __syncthreads();
    }
    bad |= given > A.c.num_pages - free_n;
    const bool any_bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.verdict = any_bad ? ATTN_ERR_BAD_SEQLENS : ATTN_OK;
  }
  // pages of the requests that shrink: several warps a request if there are few
  const int mine = cdiv(P.batch - part, A.checks), team = max(1, WARPS / max(1, mine)), teams = WARPS / team;
  bool off = false;
  for (int i = warp / team; i < mine && warp < team * teams; i += teams) {
    const int b = part + i * A.checks, n = P.seqlens[b];
    if (!evicts(A, n, P.keep[b])) continue;
    const int held = pages_of(n, shift);
    const int* table = P.block_table + b * P.table_stride;
    constexpr int U = 8;
    for (int j0 = (warp % team) * 32 + lane; j0 < held; j0 += team * 32 * U) {
      int page[U];
#pragma unroll
      for (int k = 0; k < U; ++k) page[k] = j0 + k * team * 32 < held ? __ldg(table + j0 + k * team * 32) : 0;
#pragma unroll
      for (int k = 0; k < U; ++k) off |= page[k] < 0 || page[k] >= A.c.num_pages;
    }
  }
  const bool any_off = __syncthreads_or(off);
  if (threadIdx.x == 0) A.off[part] = any_off;
}

// ONE: clusters of one CTA.
template <bool ONE>
__global__ void __launch_bounds__(ONE ? ONE_THREADS : MANY_THREADS, ONE ? 2 : 1) select_kernel(const __grid_constant__ Args A) {
  constexpr int THREADS = ONE ? ONE_THREADS : MANY_THREADS;
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(16) int s_hist[BINS];
  __shared__ int s_scratch[2][MAX_WARPS];
  __shared__ int s_found[2], s_sum[3];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const attn_kv_evict_params& P = A.p;
  const int tid = threadIdx.x, rank = ONE ? 0 : rank_of(), heads = A.c.hkv;
  const int cluster = ONE ? 1 : A.cluster, job = blockIdx.x / cluster;
  if (job >= P.batch * heads) {
    const int part = blockIdx.x - P.batch * heads * cluster;
    if (part < A.checks) check_call<THREADS>(A, part, s_scratch[0]);
    return;
  }
  const int b = job / heads, h = job - b * heads;
  const int n = P.seqlens[b], keep = P.keep[b];
  if (!evicts(A, n, keep) || keep == 0) return;         // the same for the whole cluster
  const int shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int per = cdiv(n, cluster), lo = min(rank * per, n), mine = min(per, n - lo);
  uint32_t* keys = A.keys ? A.keys + (long long)job * A.max_k + lo : s_keys;
  const int* table = P.block_table + b * P.table_stride;
  const long long recent = (long long)n + P.position_offsets[b] - P.recent;
  auto fill = [&](bool protected_only) {
    constexpr int U = 8;                                 // rows of a thread on their way together
    for (int i0 = tid; i0 < mine; i0 += THREADS * U) {
      int page[U], pos[U];
      float w[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * THREADS;
        page[k] = i < mine ? __ldg(table + ((lo + i) >> shift)) : -1;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool in = page[k] >= 0 && page[k] < A.c.num_pages;
        const long long at = (((long long)page[k] * heads + h) << shift) + ((lo + i0 + k * THREADS) & in_page);
        pos[k] = in ? __ldg(P.weights.position + at) : 0;
        w[k] = in ? __ldg(P.weights.weight + at) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * THREADS;
        const bool first = pos[k] < P.sink || pos[k] >= recent;
        const uint32_t by_weight = key_of(w[k]);
        if (i < mine) keys[i] = protected_only ? (first ? by_weight : 0) : first ? FIRST : by_weight;
      }
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
    owners_sync<ONE>();
    // bins from the top: of the first BINS / 4 threads, thread t has four
    constexpr int PER = 4;
    static_assert(BINS / PER <= THREADS, "a vector per thread");
    int sum, total;
    const int top = max(PER - 1, BINS - 1 - tid * PER);
    int4 v = make_int4(0, 0, 0, 0);
    if (ONE) {
      if (tid < BINS / PER) v = *reinterpret_cast<const int4*>(&s_hist[top - 3]);
    } else if (tid < BINS / PER) {
      // eight ranks' words on their way together (another CTA's memory is a microsecond away)
      for (int r0 = 0; r0 < cluster; r0 += 8) {
        int4 x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) x[r] = r0 + r < cluster ? peek4(&s_hist[top - 3], r0 + r) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) v = make_int4(v.x + x[r].x, v.y + x[r].y, v.z + x[r].z, v.w + x[r].w);
      }
    }
    const int bin[PER] = {v.w, v.z, v.y, v.x};
    sum = v.x + v.y + v.z + v.w;
    int before = block_before<THREADS>(sum, s_scratch[pass & 1], &total);
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
    owners_sync<ONE>();                                      // also: the histograms have been read
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
  int ties = block_before<THREADS>(equal, s_scratch[1], &total);
  // sums of the CTAs before this one: a lane reads one CTA's
  auto ranks_before = [&](int which) {
    const int x = (tid & 31) < rank ? peek(&s_sum[which], tid & 31) : 0;
    return __reduce_add_sync(0xffffffffu, x);
  };
  if (!ONE) {
    if (tid == 0) s_sum[0] = total;
    owners_sync<ONE>();
    ties += ranks_before(0);
  }
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
  const int holes0 = block_before<THREADS>(holes, s_scratch[0], &total_holes);
  __syncthreads();
  const int fills0 = block_before<THREADS>(fills, s_scratch[1], &total_fills);
  holes = holes0;
  fills = fills0;
  if (!ONE) {
    if (tid == 0) {
      s_sum[1] = total_holes;
      s_sum[2] = total_fills;
    }
    owners_sync<ONE>();
    holes += ranks_before(1);
    fills += ranks_before(2);
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
  if (!ONE) owners_sync<ONE>();                          // no CTA leaves while others read its shared memory
}

// 16 e4m3 values times 2^shift, shift < 0, rounded again.  In fp16: the product is exact
// as far as 2^-24, far below half of e4m3's least value, 2^-10; a factor below fp16's
// least number is 0, and so are its products in e4m3.
__device__ __forceinline__ uint4 times(const uint4& x, int shift) {
  const __half2 f = __float2half2_rn(exp2_int(shift));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo = e4m3x2_to_h2((uint16_t)w[j]), hi = e4m3x2_to_h2((uint16_t)(w[j] >> 16));
    *reinterpret_cast<__half2*>(&lo) = __hmul2(*reinterpret_cast<__half2*>(&lo), f);
    *reinterpret_cast<__half2*>(&hi) = __hmul2(*reinterpret_cast<__half2*>(&hi), f);
    q[j] = __byte_perm(h2_to_e4m3x2(lo), h2_to_e4m3x2(hi), 0x5410);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

// Rows [0, rows) of a page's head, one side of the cache, at a scale 2^-shift times as
// large, by one warp.  Holes among them are filled after this.
template <int D>
__device__ __forceinline__ void round_again(uint8_t* page, long long stride, int rows, int shift) {
  constexpr int PER = D / 16, N = 4;
  for (int i0 = threadIdx.x & 31; i0 < rows * PER; i0 += 32 * N) {
    uint4 x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + 32 * k;
      if (i < rows * PER) x[k] = *reinterpret_cast<const uint4*>(page + (i / PER) * stride + (i % PER) * 16);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + 32 * k;
      if (i < rows * PER) *reinterpret_cast<uint4*>(page + (i / PER) * stride + (i % PER) * 16) = times(x[k], shift);
    }
  }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(MOVE_THREADS, 3) move_kernel(const __grid_constant__ Args A) {
  __shared__ int s_page[CHUNK];              // of what fills a hole
  __shared__ int s_rows[CHUNK];              // its row in the page, the hole's in the chunk, exponents of its page
  __shared__ int s_dst[CHUNK_PAGES];         // pages of the chunk
  __shared__ int s_old[2][CHUNK_PAGES], s_new[2][CHUNK_PAGES];   // their exponents: K, V
  __shared__ int s_back[MOVE_WARPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const attn_kv_evict_params& P = A.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int heads = A.c.hkv;
  const bool off = __syncthreads_or(tid < A.checks && A.off[tid]);
  const int verdict = *A.verdict != ATTN_OK ? *A.verdict : off ? ATTN_ERR_BAD_PAGE : ATTN_OK;
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
  const int keep = r.y, pages = pages_of(keep, shift), each = cdiv(pages, A.spread);
  const int end = min(pages, (share + 1) * each), step = CHUNK >> shift;
  const int* table = P.block_table + b * P.table_stride;
  const int* to = A.to + (long long)job * A.half;
  const int* from = A.from + (long long)job * A.half;
  const int* starts = A.holes + (long long)job * (A.pages + 1);
  uint8_t* kh = A.c.k + h * A.c.sk.h;
  uint8_t* vh = A.c.v + h * A.c.sv.h;
  for (int p0 = share * each; p0 < end; p0 += step) {
    const int np = min(step, end - p0), h0 = starts[p0], count = starts[p0 + np] - h0;
    if (count == 0) continue;
    __syncthreads();                                     // the last chunk's rows have moved
    if (tid < np) {
      const int page = table[p0 + tid];
      const long long at = (long long)page * heads + h;
      s_dst[tid] = page;
      s_old[0][tid] = s_new[0][tid] = kv_exp_of(A.c.k_exp[at]);
      s_old[1][tid] = s_new[1][tid] = kv_exp_of(A.c.v_exp[at]);
    }
    __syncthreads();
    for (int i = tid; i < count; i += MOVE_THREADS) {
      const int row = to[h0 + i] - (p0 << shift), src = from[h0 + i], page = table[src >> shift];
      const long long at = (long long)page * heads + h;
      // the page that row `keep` is in may be getting new exponents from another CTA
      int ek, ev;
      if (src >> shift == keep >> shift) {
        const int2 e = A.edge[job];
        ek = e.x, ev = e.y;
      } else {
        ek = A.c.k_exp[at], ev = A.c.v_exp[at];
      }
      ek = kv_exp_of((uint8_t)ek), ev = kv_exp_of((uint8_t)ev);
      const long long w_src = (at << shift) + (src & in_page);
      const long long w_dst = (((long long)s_dst[row >> shift] * heads + h) << shift) + (row & in_page);
      const float w = P.weights.weight[w_src];
      const int pos = P.weights.position[w_src];
      atomicMax(&s_new[0][row >> shift], ek);
      atomicMax(&s_new[1][row >> shift], ev);
      s_page[i] = page;
      s_rows[i] = (src & in_page) | row << 8 | (ek - KV_EXP_MIN) << 18 | (ev - KV_EXP_MIN) << 24;
      P.weights.weight[w_dst] = w;
      P.weights.position[w_dst] = pos;
    }
    __syncthreads();
    // pages whose scale grew
    for (int q = warp; q < 2 * np; q += MOVE_WARPS) {
      const int p = q >> 1, v = q & 1, old = s_old[v][p], now = s_new[v][p];
      if (now == old) continue;
      const int page = s_dst[p], rows = min(1 << shift, keep - ((p0 + p) << shift));
      if (v) round_again<DV>(vh + page * A.c.sv.p, A.c.sv.r, rows, old - now);
      else round_again<DQK>(kh + page * A.c.sk.p, A.c.sk.r, rows, old - now);
      if (lane == 0) (v ? A.c.v_exp : A.c.k_exp)[(long long)page * heads + h] = (uint8_t)(now + KV_EXP_BIAS);
    }
    __syncthreads();
    // the rows: a thread keeps to 16 bytes of K or V and takes every LANES-th hole
    constexpr int PK = DQK / 16, PER = PK + DV / 16, LANES = MOVE_THREADS / PER, N = 4;
    const int c = tid % PER;
    const bool v = c >= PK;
    const KvStrides& st = v ? A.c.sv : A.c.sk;
    uint8_t* base = v ? vh + (c - PK) * 16 : kh + c * 16;
    const int* now = s_new[v];
    for (int i0 = tid / PER; i0 < (tid < LANES * PER ? count : 0); i0 += LANES * N) {
      uint4 x[N];
      uint8_t* dst[N];
      int shrink[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = i0 + k * LANES;
        if (i < count) {
          const int info = s_rows[i], row = info >> 8 & (CHUNK - 1), p = row >> shift;
          x[k] = *reinterpret_cast<const uint4*>(base + s_page[i] * st.p + (info & 255) * st.r);
          dst[k] = base + s_dst[p] * st.p + (row & in_page) * st.r;
          shrink[k] = (info >> (v ? 24 : 18) & 63) + KV_EXP_MIN - now[p];
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (i0 + k * LANES < count) *reinterpret_cast<uint4*>(dst[k]) = shrink[k] == 0 ? x[k] : times(x[k], shrink[k]);
    }
  }
}

struct Layout {
  size_t off_off, off_plan, off_edge, off_holes, off_to, off_from, off_keys, total;
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
  while (L->cluster < MAX_CLUSTER && cdiv(L->max_k, L->cluster) > SHARE) L->cluster *= 2;
  L->held = cdiv(L->max_k, L->cluster) <= HELD;
  L->pages = cdiv(L->max_k, c.page_size);
  L->half = L->max_k / 2 + 1;
  const size_t jobs = (size_t)p->batch * c.nhead_kv;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  size_t o = 256;
  L->off_off = o;   o = up(o + MOVE_THREADS * sizeof(int));
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
  a.off = reinterpret_cast<int*>(w + L.off_off);
  a.checks = cdiv(p->batch, ONE_THREADS / 32) < MOVE_THREADS ? cdiv(p->batch, ONE_THREADS / 32) : MOVE_THREADS;
  a.plan = reinterpret_cast<int4*>(w + L.off_plan);
  a.edge = reinterpret_cast<int2*>(w + L.off_edge);
  a.holes = reinterpret_cast<int*>(w + L.off_holes);
  a.to = reinterpret_cast<int*>(w + L.off_to);
  a.from = reinterpret_cast<int*>(w + L.off_from);
  a.keys = L.held ? nullptr : reinterpret_cast<uint32_t*>(w + L.off_keys);
  const int jobs = p->batch * p->cache.nhead_kv;
  // about two CTAs per SM, each of a page at least
  const int share = cdiv(2 * SMS, jobs);
  a.spread = L.pages < 1 ? 1 : share < L.pages ? share : L.pages;
  const size_t smem = L.held ? (size_t)cdiv(L.max_k, L.cluster) * sizeof(uint32_t) : 0;
  const auto select = L.cluster == 1 ? select_kernel<true> : select_kernel<false>;
  if (smem > 32 * 1024 && !succeeded(cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                          (int)(HELD * sizeof(uint32_t)))))
    return ATTN_ERR_CUDA;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = L.cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((jobs + cdiv(a.checks, L.cluster)) * L.cluster);
  cfg.blockDim = dim3(L.cluster == 1 ? ONE_THREADS : MANY_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (!succeeded(cudaLaunchKernelEx(&cfg, select, a))) return ATTN_ERR_CUDA;
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
