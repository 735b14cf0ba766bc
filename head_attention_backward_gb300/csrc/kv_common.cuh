// What the paged 8-bit cache's operators share: the resolved cache, the checks
// of its arguments, and the e4m3 conversions (one PTX instruction each).
#pragma once

#include <initializer_list>

#include "common.cuh"

namespace attn {

constexpr int KV_EXP_BIAS = 127;
constexpr int KV_EXP_MIN = -30;   // scales 2^-30 .. 2^30: the ratio of two scales, times any sum of
constexpr int KV_EXP_MAX = 30;    // e4m3 products, stays inside fp32's range

struct KvStrides {
  long long p, r, h;   // bytes from page to page, row to row, head to head
};

struct KvCacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_exp;
  uint8_t* v_exp;
  KvStrides sk, sv;
  int num_pages, page_shift, hkv;
};

inline bool kv_headdims(int dqk, int dv) {
  return (dqk == 64 && dv == 64) || (dqk == 128 && dv == 128) || (dqk == 192 && dv == 128) ||
         (dqk == 256 && dv == 256);
}

constexpr int SMS = 152;   // of a GB300; splits and shares are made for them

// Grids carry twice this many (head, side) pairs in their second dimension.
constexpr int KV_MAX_HEADS = 16384;

inline int kv_page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Whether a call of the runtime succeeded.  It remembers a failure until it is asked
// for: it is asked here, so that the next call's check does not find this one's.
inline bool succeeded(cudaError_t e) {
  if (e == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

inline bool aligned_to(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A dimension with one entry never uses its stride; it gets a valid one.
inline bool kv_strides(const int64_t in[3], long long pages, long long rows, long long heads, long long d, KvStrides* s) {
  if (in[0] == 0 && in[1] == 0 && in[2] == 0) {
    *s = {rows * heads * d, heads * d, d};
    return true;
  }
  *s = {pages > 1 ? in[0] : 16, in[1], heads > 1 ? in[2] : 16};
  const long long lim = 1LL << 40;
  for (long long x : {s->p, s->r, s->h})
    if (x <= 0 || x >= lim || x % 16 != 0) return false;
  return true;
}

inline int kv_resolve(const attn_kv_cache& c, KvCacheView* out) {
  if (c.num_pages < 1 || c.nhead_kv < 1 || c.nhead_kv > KV_MAX_HEADS || c.reserved != 0) return ATTN_ERR_INVALID_ARG;
  const int shift = kv_page_shift(c.page_size);
  if (shift < 0) return ATTN_ERR_INVALID_ARG;
  if (!kv_headdims(c.d_qk, c.d_v)) return ATTN_ERR_UNSUPPORTED_HEADDIM;
  if (!c.k || !c.v || !c.k_exp || !c.v_exp || !aligned_to(c.k, 16) || !aligned_to(c.v, 16)) return ATTN_ERR_INVALID_ARG;
  if (!kv_strides(c.stride_k, c.num_pages, c.page_size, c.nhead_kv, c.d_qk, &out->sk) ||
      !kv_strides(c.stride_v, c.num_pages, c.page_size, c.nhead_kv, c.d_v, &out->sv))
    return ATTN_ERR_INVALID_ARG;
  out->k = static_cast<uint8_t*>(c.k);
  out->v = static_cast<uint8_t*>(c.v);
  out->k_exp = c.k_exp;
  out->v_exp = c.v_exp;
  out->num_pages = c.num_pages;
  out->page_shift = shift;
  out->hkv = c.nhead_kv;
  return ATTN_OK;
}

// {ignored, row, head} element strides of a packed 16-bit tensor.
inline bool packed_strides(const int64_t in[3], int heads, int dim, Strides* s) {
  if (in[0] == 0 && in[1] == 0 && in[2] == 0) {
    *s = {(long long)heads * dim, dim};
    return true;
  }
  *s = {in[1], in[2]};
  const long long lim = 1LL << 36;
  return in[1] > 0 && in[2] > 0 && in[1] < lim && in[2] < lim && in[1] % 8 == 0 && in[2] % 8 == 0;
}

// Long query segments over the cache (kv_long.cu).
struct KvLong {
  int from;               // segments of more query tokens than this
  int slots;              // most of them that q can hold; 0: the path is not used
  int group, groups;      // slots whose keys are expanded at a time, and times
  long long kpad;         // rows of a slot's keys and values
  int nsplit;             // CTAs that a query tile's keys are split over at most
  long long part_rows, slot_rows;   // of their parts: see FwdSegments
  size_t off_list, off_k, off_v, off_po, off_pml, total;   // workspace; total is 0 without slots
};
KvLong kv_long_layout(const attn_kv_fwd_params& p, int max_k);
int launch_kv_long(const attn_kv_fwd_params& p, const KvCacheView& c, const Strides& sq, const Strides& so, int max_k,
                   const KvLong& L, char* ws, cudaStream_t st);
// Status words of the long path in its part of the workspace: [slots].
inline size_t kv_long_status_offset(const KvLong& L) { return L.off_list; }

// ------------------------------------------------------------------ e4m3

// Two e4m3 bytes (low first) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint16_t x) {
  uint32_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
  return y;
}

// Two fp32 values to e4m3, to nearest even; past 448 clamped, NaN kept.
__device__ __forceinline__ uint16_t f2_to_e4m3x2(float lo, float hi) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
  return y;
}

// The same from two packed fp16 values.
__device__ __forceinline__ uint16_t h2_to_e4m3x2(uint32_t x) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(x));
  return y;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of a stored scale byte, limited to the format's range.
__device__ __forceinline__ int kv_exp_of(uint8_t b) {
  const int e = (int)b - KV_EXP_BIAS;
  return e < KV_EXP_MIN ? KV_EXP_MIN : e > KV_EXP_MAX ? KV_EXP_MAX : e;
}

}  // namespace attn
