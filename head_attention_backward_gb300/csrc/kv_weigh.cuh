// What the two kernels of attn_kv_weigh share.
#pragma once

#include "common.cuh"
#include "kv_common.cuh"

namespace attn {
namespace kvweigh {

struct Args {
  const void* q;
  const float* lse;
  Strides sq;
  const int* cu_q;
  const int* st_q;
  const int* len_k;
  const int* table;
  long long table_stride;
  const int* offsets;      // of positions, per request, or null
  const int* new_lens;     // keys new to the weights, per request, or null: see fresh
  int max_k;               // min(max_seqlen_k, max_blocks pages)
  int total_q, max_q;
  int long_from;           // segments of more tokens are the other kernel's
  int hq, g;               // query heads, per kv head
  int mask, left, right;
  int fresh;               // without new_lens: 1: the last keys of a segment are its query tokens
  float scale_log2, decay;
  int nsplit;              // most splits of a request's keys
  float* weight;           // [page][kv head][row]
  int* position;
  int* status;
  KvCacheView c;
};

struct Segment {
  int lq, lk, q0;
  int fresh;               // keys from here on start from 0
  bool bad;                // lengths outside the declared bounds: left alone
};
__device__ __forceinline__ Segment segment_of(const Args& A, int b) {
  Segment s;
  s.lq = __ldg(A.cu_q + b + 1) - __ldg(A.cu_q + b);
  s.q0 = __ldg(A.st_q + b);
  s.lk = __ldg(A.len_k + b);
  const int added = A.new_lens ? __ldg(A.new_lens + b) : A.fresh ? min(s.lq, s.lk) : 0;
  s.fresh = s.lk - added;
  s.bad = s.lq < 0 || s.lq > A.max_q || s.q0 < 0 || (long long)s.q0 + s.lq > A.total_q || s.lk < 0 || s.lk > A.max_k ||
          (s.lq > 0 && (added < 0 || added > s.lk));
  if (s.bad) s.lq = 0;
  return s;
}

__device__ __forceinline__ void report(const Args& A, int code) { atomicCAS(A.status, 0, code); }

// Keys that any of the query tokens i0 .. i1 sees, lo > hi: none.
__device__ __forceinline__ void seen_by(const MaskArgs& m, int lk, int i0, int i1, int& lo, int& hi) {
  lo = 0;
  hi = lk - 1;
  if (m.left >= 0) lo = (int)max(0ll, (long long)i0 + m.off - m.left);
  if (m.right >= 0) hi = (int)min((long long)hi, (long long)i1 + m.off + m.right);
}

// Keys of a segment whose weights change, lo > hi: none.  Those that a query sees and the
// new ones, or all if the old ones decay.
__device__ __forceinline__ void changing(const Args& A, const Segment& s, const MaskArgs& m, int& lo, int& hi) {
  seen_by(m, s.lk, 0, s.lq - 1, lo, hi);
  if (lo > hi) lo = s.lk, hi = s.lk - 1;
  if (s.fresh < s.lk) lo = min(lo, s.fresh), hi = s.lk - 1;
  if (A.decay != 1.f) lo = 0, hi = s.lk - 1;
}

// Whether token i sees key j.
__device__ __forceinline__ bool sees(const MaskArgs& m, int i, int j) {
  const long long c = (long long)i + m.off;
  return (m.left < 0 || j >= c - m.left) && (m.right < 0 || j <= c + m.right);
}

// Segments of more than a.long_from tokens, on the tensor cores (kv_weigh_tc.cu), and
// the most query heads per kv head that it takes.
int long_group(int dqk);
int launch_long(const Args& a, bool bf16, int dqk, int batch, cudaStream_t st);

}  // namespace kvweigh
}  // namespace attn
