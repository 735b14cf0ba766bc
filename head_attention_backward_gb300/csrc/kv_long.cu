// Long query segments over the paged 8-bit cache: prompts and prompt pieces.
//
// Hundreds of query rows per key make the products the bound (4 Hq d flops per
// query and key against two cache bytes per key, head and column), so they
// belong on tcgen05.  The cache's pages are first expanded to 16-bit rows in
// the workspace (every e4m3 value times a power of two is exact in bf16; in fp16 it
// is rounded to multiples of 2^-24, which changes values below 2^-21 under scales
// below 2^-15, and clamped at 65504), and the tensor-core forward of attn_fwd runs
// on them.  The expansion reads each cache byte once and writes two; the forward
// reads them back.
//
// The forward's query tiles hold tokens x heads of a group, so that a short
// segment fills its 128 rows (34 tokens of 8 heads: 3 tiles instead of 8;
// 4 prompt pieces of 1,024 tokens of 4 heads, whose causal edge is then only
// 32 tokens wide: 333 to 325 us), and where the tiles leave SMs idle their keys are
// split over CTAs (109 tokens over 5,841 keys, 4 kv heads, 3 requests: 37.7 us in
// all, 59.3 with one CTA per tile).
//
// The segments are found on the device: a setup kernel lists them in slots, so
// one call may mix long segments with the short ones of kv_fwd.cu.
#include <cmath>

#include "common.cuh"
#include "fwd_tc.cuh"
#include "kv_common.cuh"

namespace attn {
namespace kvlong {

constexpr int PAD = 128;                        // keys of a tile of the forward
constexpr size_t EXPANDED_BYTES = size_t(1) << 30;   // expanded keys and values at a time (a slot at least)
constexpr int MAX_SPLITS = 16;
constexpr int NTHREADS = 256;
constexpr int SETUP_THREADS = 256;

// Query tokens above which a segment is long.  The other path's time grows with
// tokens x group (rows of 16 that each pass over the cache), this one's hardly
// up to 128 rows, but it starts some 17 us later.  Per row and cached token of a
// kv head of 128 + 128 columns the other takes about 3.5 ps, this one per cached
// token what the other takes for some 72 rows.  Device time in us, this path / the
// other, of batch x kv heads x group, up to so many cached tokens:
//   4 x 8 x 4,  4,096:  17 tokens  47 /  42,  33:  59 /  60,  49:  55 /  82,  97:  59 / 157
//   8 x 4 x 8,  4,096:   9 tokens  42 /  41,  17:  52 /  57,  33:  51 /  85,  97:  72 / 231
//   4 x 8 x 1,  4,096:  33 tokens  45 /  26,  49:  45 /  32,  97:  45 /  43
//   1 x 8 x 4,  4,096:  33 tokens  36 /  25,  49:  36 /  41,  97:  34 /  71
//   1 x 8 x 4, 32,768:   9 tokens  90 /  51,  17:  91 /  93,  33:  92 / 136,  97: 108 / 510
//   4 x 2 x 4,  1,000:  33 tokens  27 /  13,  97:  28 /  18
// The bounds keep the rule (and with it the rounding of the weights) within sight
// of the tokens: 24 at least, 24 + 96 / group at most.
static int long_from(const attn_kv_fwd_params& p, int max_k) {
  const attn_kv_cache& c = p.cache;
  const int group = p.nhead_q / c.nhead_kv;
  const long long segments = p.total_q / 32 + 1 < p.batch ? p.total_q / 32 + 1 : p.batch;
  double keys = max_k;
  if (p.mask == ATTN_MASK_WINDOW && p.window_left >= 0 && p.window_right >= 0)
    keys = std::fmin(keys, (double)p.window_left + p.window_right + 64);
  const double work = segments * c.nhead_kv * std::fmax(keys, 1.) * (c.d_qk + c.d_v) / 256.;
  const double tokens = (72 + 17e-6 / 3.5e-12 / work) / group;
  return (int)std::fmin(std::fmax(tokens, 24.), 24 + 96 / group);
}

// Splits of a query tile's keys: the number whose waves over the SMs take the
// least time, where the tiles alone (at most: q can hold no more) would not fill
// them once.
static int splits(const attn_kv_fwd_params& p, const KvLong& L, int tok) {
  const long long by_rows = p.total_q / tok + L.slots, by_slots = (long long)L.group * cdiv(p.max_seqlen_q, tok);
  const long long ctas = p.cache.nhead_kv * (by_rows < by_slots ? by_rows : by_slots);
  if (ctas >= SMS) return 1;
  int best = 1;
  float least = 0.85f;   // a split has to gain more than the join costs
  for (int n = 2; n <= MAX_SPLITS && (n - 1) * FWD_MIN_SPLIT * FWD_TILE_ROWS < L.kpad; ++n) {
    const float cost = (float)cdiv_ll(ctas * n, SMS) / n + 0.02f * n;
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

// Per slot; every array has `slots` entries.
struct Lists {
  int* status;
  int* request;
  int* zeros;
  int* len_q;
  int* start_q;
  int* len_k;
  int* start_k;
};

static Lists lists(char* ws, const KvLong& L) {
  int* a = reinterpret_cast<int*>(ws + L.off_list);
  const size_t n = L.slots;
  return {a, a + n, a + 2 * n, a + 3 * n, a + 4 * n, a + 5 * n, a + 6 * n};
}

__global__ void __launch_bounds__(SETUP_THREADS)
    setup_kernel(const int* cu_q, const int* st_q, const int* len_k, int batch, int total_q, int max_q, int max_k,
                 int from, int slots, int group, int kpad, const Lists T) {
  __shared__ int warp_n[SETUP_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int used = 0;
  bool over = false;
  for (int base = 0; base < batch; base += SETUP_THREADS) {
    const int b = base + threadIdx.x;
    int lq = 0, q0 = 0;
    if (b < batch) {
      lq = __ldg(cu_q + b + 1) - __ldg(cu_q + b);
      q0 = __ldg(st_q + b);
      if (lq < 0 || lq > max_q || q0 < 0 || (long long)q0 + lq > total_q) lq = 0;   // reported by the other path
    }
    const bool is_long = lq > from;
    const uint32_t votes = __ballot_sync(0xffffffffu, is_long);
    if (lane == 0) warp_n[warp] = __popc(votes);
    __syncthreads();
    int at = used, all = used;
    for (int w = 0; w < SETUP_THREADS / 32; ++w) {
      if (w < warp) at += warp_n[w];
      all += warp_n[w];
    }
    at += __popc(votes & ((1u << lane) - 1));
    if (is_long && at < slots) {
      const int lk = __ldg(len_k + b);
      T.status[at] = ATTN_OK;
      T.request[at] = b;
      T.zeros[at] = 0;
      T.len_q[at] = lq;
      T.start_q[at] = q0;
      T.len_k[at] = lk < 0 ? 0 : lk > max_k ? max_k : lk;
      T.start_k[at] = (at % group) * kpad;
    }
    over |= is_long && at >= slots;   // only where segments overlap one another
    used = all;
    __syncthreads();
  }
  for (int i = (used < slots ? used : slots) + threadIdx.x; i < slots; i += SETUP_THREADS) {
    T.status[i] = ATTN_OK;
    T.request[i] = 0;
    T.zeros[i] = T.len_q[i] = T.start_q[i] = T.len_k[i] = T.start_k[i] = 0;
  }
  if (__syncthreads_or(over) && threadIdx.x == 0) T.status[0] = ATTN_ERR_BAD_SEQLENS;
}

template <typename T> struct Out2;
template <> struct Out2<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Out2<__half> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {   // finite stays finite
    const float lim = 65504.f;
    a = fabsf(a) > lim ? copysignf(lim, a) : a;
    b = fabsf(b) > lim ? copysignf(lim, b) : b;
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// 16 e4m3 values times f as 16-bit values.
template <typename T>
__device__ __forceinline__ void expand16(const uint4& x, float f, uint4* dst) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = e4m3x2_to_h2((uint16_t)w[i]), hi = e4m3x2_to_h2((uint16_t)(w[i] >> 16));
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    y[2 * i] = Out2<T>::pack(a.x * f, a.y * f);
    y[2 * i + 1] = Out2<T>::pack(b.x * f, b.y * f);
  }
  dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
  dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

// Rows [16 blockIdx.x, + 16) of a slot's keys and values (blockIdx.y: the slot
// of the group), of the forward's tiles that the segment sees; rows that it does
// not see become 0, whatever they or their pages hold.  A page outside the cache empties the segment's keys.
template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    expand_kernel(const Lists L, int slot0, const KvCacheView c, int dqk, int dv, const int* table,
                  long long table_stride, T* k16, T* v16, long long kpad, int mask, int left, int right) {
  const int slot = slot0 + blockIdx.y;
  const int lk = L.len_k[slot], lq = L.len_q[slot], row0 = blockIdx.x * 16;
  const MaskArgs m = mask_args(mask, left, right, lq, lk);
  const int klo = m.left >= 0 ? max(0, m.off - m.left) : 0;
  const int khi = m.right >= 0 ? min(lk - 1, lq - 1 + m.off + m.right) : lk - 1;
  if (row0 < klo / PAD * PAD || khi < 0 || row0 >= (khi / PAD + 1) * PAD) return;
  const bool any = row0 + 16 > klo && row0 <= khi;   // 16 rows lie in one page
  int page = 0;
  if (any) {
    page = __ldg(table + L.request[slot] * table_stride + (row0 >> c.page_shift));
    if (page < 0 || page >= c.num_pages) {
      if (threadIdx.x == 0) {
        L.len_k[slot] = 0;
        L.status[slot] = ATTN_ERR_BAD_PAGE;
      }
      return;
    }
  }
  const int in0 = row0 & ((1 << c.page_shift) - 1);
  const int pk = dqk / 16, pv = dv / 16, per = pk + pv;    // 16-byte pieces of a head's row, K then V
  const long long out0 = (long long)blockIdx.y * kpad + row0;
  for (int i = blockIdx.z * NTHREADS + threadIdx.x; i < 16 * c.hkv * per; i += NTHREADS * gridDim.z) {
    const int r = i / (c.hkv * per), x = i - r * (c.hkv * per);
    const bool is_v = x >= c.hkv * pk;
    const int y = is_v ? x - c.hkv * pk : x, n = is_v ? pv : pk;
    const int h = y / n, p = y - h * n;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float f = 1.f;
    if (any && row0 + r >= klo && row0 + r <= khi) {
      const KvStrides& s = is_v ? c.sv : c.sk;
      raw = __ldg(reinterpret_cast<const uint4*>((is_v ? c.v : c.k) + page * s.p + (in0 + r) * s.r + h * s.h + p * 16));
      f = exp2_int(kv_exp_of(__ldg((is_v ? c.v_exp : c.k_exp) + (long long)page * c.hkv + h)));
    }
    T* dst = (is_v ? v16 + ((out0 + r) * c.hkv + h) * dv : k16 + ((out0 + r) * c.hkv + h) * dqk) + p * 16;
    expand16<T>(raw, f, reinterpret_cast<uint4*>(dst));
  }
}

template <typename T>
static int launch(const attn_kv_fwd_params& p, const KvCacheView& c, const Strides& sq, const Strides& so, int max_k,
                  const KvLong& L, char* ws, cudaStream_t st) {
  const Lists T_ = lists(ws, L);
  const int* st_q = p.cu_seqlens_q_padded ? p.cu_seqlens_q_padded : p.cu_seqlens_q;
  setup_kernel<<<1, SETUP_THREADS, 0, st>>>(p.cu_seqlens_q, st_q, p.seqlens_k, p.batch, p.total_q, p.max_seqlen_q, max_k,
                                            L.from, L.slots, L.group, (int)L.kpad, T_);
  // what follows reads the lists, and each forward the keys expanded for it
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  T* k16 = reinterpret_cast<T*>(ws + L.off_k);
  T* v16 = reinterpret_cast<T*>(ws + L.off_v);
  attn_fwd_params f{};
  f.dtype = p.dtype;
  f.nhead_q = p.nhead_q;
  f.nhead_kv = p.cache.nhead_kv;
  f.seqlen_q = p.max_seqlen_q < p.total_q ? p.max_seqlen_q : p.total_q;
  f.seqlen_k = max_k;
  f.total_q = p.total_q;
  f.d_qk = p.cache.d_qk;
  f.d_v = p.cache.d_v;
  f.mask = p.mask;
  // a bound that no key is beyond is none (and keeps the forward's sums in 32 bits)
  f.window_left = p.window_left >= max_k ? -1 : p.window_left;
  f.window_right = p.window_right >= p.max_seqlen_q || p.window_right >= p.total_q ? -1 : p.window_right;
  const int left = p.mask == ATTN_MASK_WINDOW ? f.window_left : -1, right = p.mask == ATTN_MASK_WINDOW ? f.window_right : -1;
  f.softmax_scale = p.softmax_scale;
  f.q = p.q;
  f.k = k16;
  f.v = v16;
  f.o = p.o;
  f.lse = p.lse;
  FwdLayout lay{};
  lay.q = sq;
  lay.o = so;
  lay.k = {(long long)f.nhead_kv * f.d_qk, f.d_qk};
  lay.v = {(long long)f.nhead_kv * f.d_v, f.d_v};
  lay.hq0 = p.nhead_q;
  for (int g = 0; g < L.groups; ++g) {
    const int s0 = g * L.group, n = s0 + L.group <= L.slots ? L.group : L.slots - s0;
    // few rows: their pieces over more CTAs (3 segments of 600
    // tokens, 8 heads: 6.0 us against 9.7)
    const long long ctas = L.kpad / 16 * n;
    const int rounds = cdiv(16 * f.nhead_kv * (f.d_qk + f.d_v) / 16, NTHREADS);
    const int full = 8 * SMS;   // CTAs that an SM holds
    const int share = ctas >= full ? 1 : (int)(full / ctas < rounds ? full / ctas : rounds);
    if (max_k > 0)
      expand_kernel<T><<<dim3((unsigned)(L.kpad / 16), n, share), NTHREADS, 0, st>>>(T_, s0, c, f.d_qk, f.d_v, p.block_table,
                                                                             p.table_stride, k16, v16, L.kpad, f.mask,
                                                                             left, right);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
    f.batch = n;
    f.total_k = (int)(n * L.kpad);
    const FwdSegments seg{T_.zeros + s0, T_.len_q + s0, T_.start_q + s0, T_.len_k + s0, T_.start_k + s0, L.nsplit,
                          L.part_rows, L.slot_rows, reinterpret_cast<float*>(ws + L.off_po), reinterpret_cast<float2*>(ws + L.off_pml),
                          T_.status + s0};
    const int r = launch_fwd_tc(f, lay, st, &seg);
    if (r != ATTN_OK) return r;
  }
  return ATTN_OK;
}

}  // namespace kvlong

KvLong kv_long_layout(const attn_kv_fwd_params& p, int max_k) {
  KvLong L{};
  L.from = 0x7fffffff;
  const attn_kv_cache& c = p.cache;
  const int group = p.nhead_q / c.nhead_kv;
  const bool built = c.d_qk <= 192 && p.softmax_scale > 0.f && group <= FWD_TILE_ROWS;
  const int from = kvlong::long_from(p, max_k);
  if (!built || p.max_seqlen_q <= from) return L;
  L.from = from;
  // segments of more than `from` rows that do not overlap
  const long long fit = p.total_q / (from + 1);
  L.slots = (int)(fit < p.batch ? fit : p.batch);
  if (L.slots == 0) return L;
  L.kpad = cdiv_ll(max_k > 0 ? max_k : 1, kvlong::PAD) * kvlong::PAD;
  const size_t row = (size_t)c.nhead_kv * (c.d_qk + c.d_v) * 2;
  long long g = (long long)(kvlong::EXPANDED_BYTES / (row * L.kpad));
  g = g < 1 ? 1 : g > L.slots ? L.slots : g;
  g = g * L.kpad > (1LL << 30) ? (1LL << 30) / L.kpad : g;   // rows stay 32-bit coordinates
  L.group = (int)(g < 1 ? 1 : g > 65535 ? 65535 : g);
  L.groups = cdiv(L.slots, L.group);
  L.nsplit = kvlong::splits(p, L, FWD_TILE_ROWS / group);
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  size_t o = 0;
  L.off_list = o;
  o = up(o + (size_t)L.slots * 7 * sizeof(int));
  L.off_k = o;
  o = up(o + (size_t)L.group * L.kpad * c.nhead_kv * c.d_qk * 2);
  L.off_v = o;
  o = up(o + (size_t)L.group * L.kpad * c.nhead_kv * c.d_v * 2);
  L.slot_rows = p.max_seqlen_q < p.total_q ? p.max_seqlen_q : p.total_q;
  if (L.slot_rows * L.group >= p.total_q) L.slot_rows = 0;
  L.part_rows = L.slot_rows ? L.slot_rows * L.group : p.total_q;
  const size_t parts = L.nsplit > 1 ? (size_t)L.nsplit * L.part_rows * p.nhead_q : 0;
  L.off_po = o;
  o = up(o + parts * c.d_v * sizeof(float));
  L.off_pml = o;
  o = up(o + parts * sizeof(float2));
  L.total = o;
  return L;
}

int launch_kv_long(const attn_kv_fwd_params& p, const KvCacheView& c, const Strides& sq, const Strides& so, int max_k,
                   const KvLong& L, char* ws, cudaStream_t st) {
  if (p.dtype == ATTN_BF16) return kvlong::launch<__nv_bfloat16>(p, c, sq, so, max_k, L, ws, st);
  return kvlong::launch<__half>(p, c, sq, so, max_k, L, ws, st);
}

}  // namespace attn
