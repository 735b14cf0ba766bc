// Bookkeeping of a serving step (attn_kv_plan): prefix sums over the requests,
// a stack of free pages, one slot and position per new token.
//
// A few kilobytes move, so the call is its launch and dependent trips to memory:
// the lengths, then the stack and tables (first to check them, then, out of L1,
// to use them).  Slots are worked out from what was read, not from the entries
// just written, so nothing waits for a store.  One CTA does it all: the sums of a
// batch of 8192 requests are 17 requests per thread, and nothing has to wait for
// another CTA.  Only the slots and positions of many tokens (prompts) are left to
// a second kernel that spreads them over the GPU, launched early so that it waits
// in place.
#include "common.cuh"
#include "kv_common.cuh"

namespace attn {
namespace kvplan {

// One request per thread up to 256; more threads make every barrier slower than
// they make the loops shorter (256 requests of a token each: 4.3 us with 256, 4.7 with 512, 6.5 with
// 1,024; 512: 5.3, 4.8, 6.6; 8,000: 18.9, 14.2, 13.7).
constexpr int MAX_THREADS = 512;
constexpr int SMALL_THREADS = 256;
constexpr int FILL_THREADS = 256;
// Tokens from which a second kernel writes them (2,000: 7.8 us with it, 8.9 without; 4,000:
// 8.0 and 14.0; 700: 4.8 and 3.8).
constexpr int FILL_FROM = 1024;

struct Sums {
  long long tok, take, back;
};

__device__ __forceinline__ Sums add(Sums a, Sums b) { return {a.tok + b.tok, a.take + b.take, a.back + b.back}; }

// Largest b with prefix[b] <= x, for prefix[0] = 0 <= x < prefix[n]; three
// probes at a time, since each step waits for shared memory.
__device__ __forceinline__ int find(const int* prefix, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 3) >> 2, a = lo + step, b = min(a + step, hi), c = min(b + step, hi);
    const bool pa = prefix[a] <= x, pb = prefix[b] <= x, pc = prefix[c] <= x;
    lo = pc ? c : pb ? b : pa ? a : lo;
    hi = pc ? hi : pb ? c : pa ? b : a;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((long long)tokens + (1 << shift) - 1) >> shift); }

__global__ void __launch_bounds__(MAX_THREADS) plan_kernel(const attn_kv_plan_params P, const int shift, const bool fill) {
  extern __shared__ int sm[];
  const int n = P.batch;
  int* cu = sm;                   // [n + 1] new tokens before request b
  int* take = cu + n + 1;         // [n + 1] pages popped before it
  int* back = take + n + 1;       // [n + 1] pages given back before it
  int* len0 = back + n + 1;       // [n]     tokens it keeps
  __shared__ Sums part[MAX_THREADS / 32];
  const int threads = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!fill) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = cdiv(n, threads) | 1;   // odd: the threads' entries lie in different banks
  const int b0 = min(tid * per, n), b1 = min(b0 + per, n);
  const int free_n = *P.free_count;   // the output may be the same word: read by all before the first barrier
  const long long cap = (long long)P.max_blocks << shift;
  auto outside = [&](int page) { return page < 0 || page >= P.num_pages; };
  bool bad = free_n < 0 || free_n > P.num_pages, off = false;
  int filled = 0;
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int add_n = P.new_lens[b], len = P.seqlens[b];
    if (add_n < ATTN_KV_RELEASE || len < 0 || len > cap || (add_n > 0 && (long long)len + add_n > cap)) {
      bad = true;
      continue;
    }
    const int held = pages_of(len, shift);
    if (add_n == ATTN_KV_RELEASE) {
      mine.back += held;
    } else {
      mine.tok += add_n;
      mine.take += pages_of(len + add_n, shift) - held;
      // the page that the new tokens fill up first; looked at below, where it has arrived
      if (add_n > 0 && (len & ((1 << shift) - 1))) {
        off |= outside(filled);
        filled = P.block_table[b * P.table_stride + held - 1];
      }
    }
  }
  // exclusive prefix over the threads
  Sums s = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    Sums o;
    o.tok = __shfl_up_sync(0xffffffffu, s.tok, d);
    o.take = __shfl_up_sync(0xffffffffu, s.take, d);
    o.back = __shfl_up_sync(0xffffffffu, s.back, d);
    if (lane >= d) s = add(s, o);
  }
  if (lane == 31) part[warp] = s;
  const bool any_bad = __syncthreads_or(bad);
  Sums before{0, 0, 0}, total{0, 0, 0};
  for (int w = 0; w < threads / 32; ++w) {
    if (w == warp) before = total;
    total = add(total, part[w]);
  }
  before = add(before, Sums{s.tok - mine.tok, s.take - mine.take, s.back - mine.back});
  int why = any_bad || total.tok > P.max_tokens || total.back > P.num_pages - free_n ? ATTN_ERR_BAD_SEQLENS
            : total.take > free_n + total.back                                       ? ATTN_ERR_OUT_OF_PAGES
                                                                                     : ATTN_OK;
  if (why == ATTN_OK) {
    // the sums fit 32 bits from here on
    for (int b = b0; b < b1; ++b) {
      const int add_n = P.new_lens[b], len = P.seqlens[b];
      cu[b] = (int)before.tok;
      take[b] = (int)before.take;
      back[b] = (int)before.back;
      const int held = pages_of(len, shift);
      if (add_n == ATTN_KV_RELEASE) {
        len0[b] = 0;
        before.back += held;
      } else {
        len0[b] = len;
        before.tok += add_n;
        before.take += pages_of(len + add_n, shift) - held;
      }
    }
    if (tid == 0) {
      cu[n] = (int)total.tok;
      take[n] = (int)total.take;
      back[n] = (int)total.back;
    }
  }
  __syncthreads();
  const int nback = why == ATTN_OK ? back[n] : 0, ntake = why == ATTN_OK ? take[n] : 0;
  const int top = free_n + nback;
  // page number i given back / popped i-th (before anything is written)
  auto given = [&](int i) {
    const int b = find(back, n, i);
    return P.block_table[b * P.table_stride + (i - back[b])];
  };
  auto popped = [&](int i) {
    const int at = top - 1 - i;
    return at < free_n ? P.free_pages[at] : given(at - free_n);
  };
  off |= outside(filled);
  for (int i = tid; i < nback; i += threads) off |= outside(given(i));
  for (int i = tid; i < ntake; i += threads) {
    const int at = top - 1 - i;
    if (at < free_n) off |= outside(P.free_pages[at]);
  }
  if (__syncthreads_or(off)) why = ATTN_ERR_BAD_PAGE;
  if (why != ATTN_OK) {
    for (int b = tid; b <= n; b += threads) {
      P.cu_seqlens[b] = 0;
      if (b < n) P.seqlens_out[b] = P.seqlens[b];
    }
    for (int t = tid; fill && t < P.max_tokens; t += threads) {
      P.positions[t] = 0;
      P.slots[t] = -1;
    }
    if (tid == 0) {
      *P.free_count_out = free_n;
      *P.status = why;
    }
    return;
  }
  // No entry written here is read here: pushes land above free_n, pops in
  // entries past the pages a request holds.
  for (int i = tid; i < nback; i += threads) P.free_pages[free_n + i] = given(i);
  for (int i = tid; i < ntake; i += threads) {
    const int b = find(take, n, i);
    P.block_table[b * P.table_stride + pages_of(len0[b], shift) + (i - take[b])] = popped(i);
  }
  for (int b = tid; b <= n; b += threads) {
    P.cu_seqlens[b] = cu[b];
    if (b < n) P.seqlens_out[b] = len0[b] + cu[b + 1] - cu[b];
  }
  if (tid == 0) {
    *P.free_count_out = top - ntake;
    *P.status = ATTN_OK;
  }
  if (!fill) return;
  const int total_tok = cu[n];
  for (int t = tid; t < P.max_tokens; t += threads) {
    int pos = 0;
    long long slot = -1;
    if (t < total_tok) {
      const int b = find(cu, n, t);
      pos = len0[b] + t - cu[b];
      const int block = pos >> shift, held = pages_of(len0[b], shift);
      const int page = block < held ? P.block_table[b * P.table_stride + block] : popped(take[b] + block - held);
      slot = ((long long)page << shift) + (pos & ((1 << shift) - 1));
    }
    P.positions[t] = pos;
    P.slots[t] = slot;
  }
}

// Positions and slots from what plan_kernel wrote (no tokens where it refused).
__global__ void __launch_bounds__(FILL_THREADS) fill_kernel(const attn_kv_plan_params P, const int shift) {
  extern __shared__ int cu[];     // [batch + 1]
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = P.batch;
  for (int b = threadIdx.x; b <= n; b += FILL_THREADS) cu[b] = __ldcg(P.cu_seqlens + b);
  __syncthreads();
  const int t = blockIdx.x * FILL_THREADS + threadIdx.x;
  if (t >= P.max_tokens) return;
  int pos = 0;
  long long slot = -1;
  if (t < cu[n]) {
    const int b = find(cu, n, t);
    pos = __ldcg(P.seqlens_out + b) - cu[b + 1] + t;
    const int page = __ldcg(P.block_table + b * P.table_stride + (pos >> shift));
    slot = ((long long)page << shift) + (pos & ((1 << shift) - 1));
  }
  P.positions[t] = pos;
  P.slots[t] = slot;
}

// Shared memory of plan_kernel's four arrays.
static size_t plan_smem(int batch) { return (4 * (size_t)batch + 3) * sizeof(int); }

static int run(const attn_kv_plan_params* p, cudaStream_t st) {
  if (!p || p->reserved != 0) return ATTN_ERR_INVALID_ARG;
  const int shift = kv_page_shift(p->page_size);
  if (shift < 0 || p->batch < 1 || p->batch > ATTN_KV_MAX_BATCH || p->num_pages < 1 || p->max_blocks < 1 ||
      p->max_tokens < 0 || p->max_tokens > (1 << 30))
    return ATTN_ERR_INVALID_ARG;
  if (((long long)p->max_blocks << shift) > (1LL << 30) || p->table_stride < p->max_blocks ||
      p->table_stride >= (1LL << 36))
    return ATTN_ERR_INVALID_ARG;
  const void* need[] = {p->new_lens, p->seqlens, p->seqlens_out, p->block_table, p->free_pages, p->free_count,
                        p->free_count_out, p->cu_seqlens, p->status};
  for (const void* x : need)
    if (!x || !aligned_to(x, 4)) return ATTN_ERR_INVALID_ARG;
  if (p->max_tokens > 0 && (!p->positions || !p->slots)) return ATTN_ERR_INVALID_ARG;
  if (!aligned_to(p->positions, 4) || !aligned_to(p->slots, 8)) return ATTN_ERR_INVALID_ARG;
  // The default limit is 48 KB less the static shared memory.  The limit is the
  // kernel's, not the call's: always the same one, so that a call on another thread
  // cannot lower it before the launch.
  const size_t smem = plan_smem(p->batch);
  if (smem > 32 * 1024 && !succeeded(cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                          (int)plan_smem(ATTN_KV_MAX_BATCH))))
    return ATTN_ERR_CUDA;
  const bool fill = p->max_tokens <= FILL_FROM;
  const int threads = p->batch <= SMALL_THREADS ? SMALL_THREADS : MAX_THREADS;
  plan_kernel<<<1, threads, smem, st>>>(*p, shift, fill);
  // the second kernel reads what the first wrote: never without it
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (!fill) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cdiv(p->max_tokens, FILL_THREADS));
    cfg.blockDim = dim3(FILL_THREADS);
    cfg.dynamicSmemBytes = (p->batch + 1) * sizeof(int);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    if (!succeeded(cudaLaunchKernelEx(&cfg, fill_kernel, *p, shift))) return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

}  // namespace kvplan
}  // namespace attn

extern "C" int attn_kv_plan(const attn_kv_plan_params* p, cudaStream_t stream) { return attn::kvplan::run(p, stream); }
