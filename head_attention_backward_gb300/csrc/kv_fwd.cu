// Attention of packed query segments over the paged 8-bit cache (attn_kv_fwd).
//
//   O = softmax(s Q K^T) V,  K = 2^ek Kq, V = 2^ev Vq per page and kv head.
//
// Decoding reads every visible cache byte once and does 4 Hq / Hkv flops per
// byte: bound by memory, far from the tensor cores' rate.  So the query rows
// that share a kv head (tokens x Hq / Hkv, in tiles of 8 or 16) meet the cache
// in warp-level m16n8k16 products, and the work is laid out for the loads:
//
// * A CTA owns one row tile, one kv head and one split of the keys; its four
//   warps take 16-key tiles in turn, each with a ring of its own that its lane
//   0 keeps full by TMA (a 16-row box of a page and head, swizzled).  No
//   barrier joins the warps until the end.  A tile lies in one page, so its
//   scales are uniform.
// * The products are transposed, S^T = K Q^T and O^T = V^T P^T: the 16-row side
//   of the instruction holds keys and value columns, the 8-column side the few
//   query rows.  S^T becomes the operand P^T by one 8 x 8 transposition per
//   eight keys inside the warp.
// * e4m3 is exact in fp16.  The contraction's order is free, so a lane takes
//   16 consecutive bytes of a K row as its share of four k-steps and 16
//   consecutive bytes of four V rows as its share of eight column tiles: wide
//   shared loads, one conversion per two values.  So is the order of the keys:
//   key_of() pairs rows so that the swizzle keeps both kinds of load free of
//   bank conflicts (of V at head dim 64, two-way).
// * q goes to fp16 under a power-of-two scale per row (largest magnitude in
//   [2^14, 2^15)), which is exact for bf16 too unless an element is 2^-28 of
//   its row's largest.  P is fp16 with its running maximum at 2^4: 11 bits down
//   to 2^-18 of the row's maximum, 2^-28 reached.  Scores, maxima, sums and O
//   are fp32.
// * The accumulator is held in units of one V scale; a page whose scale is
//   within 2^4 of it has their ratio r put on P before its one rounding, others
//   move the unit.  Such a P has 11 bits down to 2^-18 / r and reaches 2^-28 / r
//   of the row's maximum: r = 2^-4 at worst, 2^-14 and 2^-24.
//
// In small grids the splits of a row tile form a thread-block cluster and are
// joined through its shared memory; otherwise they leave (O, max, sum) in the
// workspace, where a second small kernel joins them.  The order is fixed.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kv_common.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace kvfwd {

constexpr int NWARPS = 4;
constexpr int NTHREADS = 32 * NWARPS;
constexpr int TILE = 16;            // keys of a warp's step
constexpr int META_TILES = 256;     // tiles whose pages are held in shared memory at a time
// Splits.  A job is one row tile of one request and kv head.  The host sets how
// many splits a job has at most, the device how long they are, from the request's
// own length, so that max_seqlen_k need not be tight.
// * Few jobs (at most half a wave): splits for one wave.  Of one request, all
//   equal: two CTAs per SM (131,072 tokens, 8 kv heads: 50.5 us with 304 CTAs, 55.3
//   with 152, 56.3 with 608: more parts to join).  Of several, whose lengths differ:
//   as many as are resident (head dim 128, four per SM: 4 requests of up to 16,384
//   tokens: 21.2 us with 608 CTAs, 29.1 with 304, 24.5 with 912; 16 of up to 2,000:
//   14.6, 17.8 and 20.5.  Head dim 192, three: 29.8 us with 456 CTAs, 30.7 with 608;
//   16.4 and 20.2.  Head dim 256, two: 8 of up to 1,000 11.4 us with 304, 19.0 with 608).
// * Many jobs: at most MAX_GRID CTAs, which still evens out ragged lengths (64
//   requests of up to 8,192 tokens: 110.2 us, with 4,608 CTAs 108.9, with one or two
//   splits 114); the CTAs without work behind a loose bound cost little (64
//   requests of up to 1,000 tokens: 22.4 us under a bound of 1,000, 28.6 under one of
//   131,072; with 4,608 CTAs 34.7).
// * None so short that its prologue outweighs it (4 requests of 1,000 tokens: 8.5
//   us at 12 tiles, 8.8 at 8, 8.9 at 16).
// A list of (job, split) items made on the device by a kernel before this one, and
// taken by persistent CTAs, was slower throughout (65 us, 119 us and 32 us in these
// cases): it puts two more trips to memory in front of the first load.
constexpr int HALF_WAVE = 2 * SMS;
constexpr int MAX_GRID = 2560;
constexpr int EVEN_TILES = 64;
constexpr int MIN_TILES = 12;
// Up to eight splits in a grid of one wave are joined as clusters: no second
// launch, 8.5 us against 9.2 in that last case.  Not in larger grids, where the
// CTAs of a cluster hold their SMs for its slowest (158 us against 108 for the 64
// requests), nor where the clusters that fit next to each other are fewer than the
// jobs (54 of eight splits, three CTAs per SM: 16.8 us, 10.6 without).
constexpr int MAX_CLUSTER = 8;
constexpr int EV_SLACK = 4;         // V scales within 2^4 of the accumulator's unit go on P
constexpr float P_LOG2 = 4.f;       // P = 2^4 at the running maximum
constexpr float SLACK_LOG2 = 7.f;   // growth of the maximum that is let pass: P <= 2^(4 + 7 + 4)

// CTAs per SM that the registers have to allow (shared memory allows them too).
constexpr int resident(int dqk, int nt) { return (dqk == 256 ? 3 : dqk == 192 ? 4 : 5) - nt; }

// NT: query rows of a CTA in units of 8.
template <int DQK, int DV, int NT>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int KB = TILE * DQK, VB = TILE * DV;
  static constexpr int STAGE = KB + VB;
  static constexpr int NST = STAGE <= 2048 ? 6 : 3;
  static constexpr int RING = NST * STAGE;
  static constexpr int OFF_BAR = NWARPS * RING;                        // uint64_t[NWARPS][NST]
  static constexpr int OFF_META = OFF_BAR + NWARPS * NST * 8;          // int2[META_TILES + 1]: page, exponents
  static constexpr int OFF_ML = OFF_META + (META_TILES + 1) * 8;       // float[2][NWARPS][ROWS]
  static constexpr int SMEM = OFF_ML + 2 * NWARPS * ROWS * 4 + ROWS * 8 + 8 + 1024;   // + alignment slack
  static constexpr int RESIDENT = resident(DQK, NT);
  static constexpr int OFF_JOIN = NWARPS * ROWS * DV * 4;              // float[ROWS][DV], behind the warps' parts
  static_assert(OFF_JOIN + ROWS * DV * 4 <= NWARPS * RING, "the joins reuse the rings");
};

struct Maps {
  CUtensorMap k, v;      // (d, heads, rows of a page, pages)
};

struct Args {
  const void* q;
  void* o;
  float* lse;
  Strides sq, so;
  const int* cu_q;
  const int* st_q;
  const int* len_k;
  const int* table;
  long long table_stride;
  int max_k;             // min(max_seqlen_k, max_blocks pages)
  int total_q, max_q, batch;
  int long_from;         // segments of more tokens are left to the long path
  int hq, g;             // query heads, per kv head
  int mask, left, right;
  float scale_log2;
  int nsplit, min_tiles, mtiles;   // most splits of a job, least tiles of one; most row tiles of a request: see slot_of
  int direct;            // 1: slots are request x row tile
  int cluster;           // 1: the splits of a job are a cluster
  int job_rows;          // most rows that a row tile can have
  float* part_o;         // [job][nsplit][job_rows][DV]
  float2* part_ml;       // [job][nsplit][job_rows]
  int* status;           // one per CTA: what its lengths, pages and loads gave
  KvCacheView c;
};

// What a request's row tile and the keys it sees come to.
struct Job {
  int lq, lk, q0;        // segment
  int row0, nrow;        // rows of the tile (row = token * g + head of the group)
  int klo, khi;          // keys that any of its rows sees, khi < klo: none
  int kbeg;              // klo rounded down to a tile
  int ntile;
  bool bad;              // lengths outside the declared bounds
};

template <int ROWS>
__device__ __forceinline__ Job make_job(const Args& A, int b, int m, MaskArgs& mk) {
  Job j;
  const int a = __ldg(A.cu_q + b);
  j.lq = __ldg(A.cu_q + b + 1) - a;
  j.q0 = __ldg(A.st_q + b);
  j.lk = __ldg(A.len_k + b);
  j.bad = j.lq < 0 || j.lq > A.max_q || j.q0 < 0 || (long long)j.q0 + j.lq > A.total_q;
  if (j.bad || j.lq > A.long_from) j.lq = 0;
  if (j.lk < 0 || j.lk > A.max_k) {
    j.bad = true;
    j.lk = j.lk < 0 ? 0 : A.max_k;
  }
  mk = mask_args(A.mask, A.left, A.right, j.lq, j.lk);
  j.row0 = m * ROWS;
  j.nrow = min(ROWS, j.lq * A.g - j.row0);
  j.klo = 0;
  j.khi = j.lk - 1;
  if (j.nrow > 0) {
    const int i0 = j.row0 / A.g, i1 = (j.row0 + j.nrow - 1) / A.g;
    if (mk.left >= 0) j.klo = (int)max(0ll, (long long)i0 + mk.off - mk.left);
    if (mk.right >= 0) j.khi = (int)min((long long)j.khi, (long long)i1 + mk.off + mk.right);
  }
  j.kbeg = j.klo & ~(TILE - 1);
  j.ntile = j.khi >= j.klo ? (j.khi - j.kbeg) / TILE + 1 : 0;
  return j;
}

// Request and row tile of a slot.  Where requests may have many more row tiles than
// q has rows, the grid follows the packed rows (64 single tokens of 4 heads per kv
// head under a max_seqlen_q of 32: 640 jobs, not 4,096; 132 us, not 181): request
// b's tiles start at slot cu_q[b] g / ROWS + b, which leaves room for them.  A warp
// searches 32 requests at a time.
struct Slot {
  int b, m;
};
template <int ROWS>
__device__ __forceinline__ Slot slot_of(const Args& A, int slot) {
  if (A.direct) return {slot / A.mtiles, slot % A.mtiles};
  const int lane = threadIdx.x & 31;
  const long long c0 = __ldg(A.cu_q);
  auto first = [&](int i) { return (__ldg(A.cu_q + i) - c0) * A.g / ROWS + i; };
  int lo = 0, hi = A.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const uint32_t at = __ballot_sync(0xffffffffu, i < hi && first(i) <= slot);
    const int n = at == 0xffffffffu ? 32 : __ffs(~at) - 1;   // probes up to the first beyond the slot
    hi = min(hi, lo + (n + 1) * step);
    lo += n * step;
  }
  const long long m = slot - first(lo);
  return {lo, m >= 0 && m < (1 << 26) ? (int)m : 1 << 26};   // past any row
}
// Whether a request's lengths are wrong that no slot may lead to: a search over
// offsets that go back misses some.
template <int ROWS>
__device__ __forceinline__ bool misses(const Args& A, int slot) {
  MaskArgs mk;
  return !A.direct && slot < A.batch &&
         (make_job<ROWS>(A, slot, 0, mk).bad || (long long)__ldg(A.cu_q + A.batch) - __ldg(A.cu_q) > A.total_q);
}

// Tiles of a job's splits: equal shares, whole turns of the warps.
__device__ __forceinline__ int split_tiles(const Args& A, const Job& j) {
  return cdiv(max(A.min_tiles, cdiv(j.ntile, A.nsplit)), NWARPS) * NWARPS;
}

__device__ __forceinline__ bool sees(const MaskArgs& m, int i, int j) {
  const long long c = (long long)i + m.off;
  return (m.left < 0 || j >= c - m.left) && (m.right < 0 || j <= c + m.right);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* desc, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(desc)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Bounded wait; a tile that does not arrive within the limit ends the loop.
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 20000))
    if (ptx::globaltimer() - t0 > WAIT_LIMIT_NS) return false;
  return true;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  return ptx::mbar_try_wait(bar, parity) || wait_slow(bar, parity);
}

// Cluster of the splits: barrier, and reads of another CTA's shared memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t in_cta(uint32_t smem_addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Byte offset of 16-byte piece c of row r in a warp's K or V tile: boxes of 16
// rows of 128 bytes (64 where D is no multiple of 128), with the swizzle of
// that width as TMA writes it.
template <int D>
struct Box {
  static constexpr int W = D % 128 == 0 ? 128 : 64;
  static constexpr int N = D / W;
};
template <int D>
__device__ __forceinline__ int off(int r, int c) {
  if (Box<D>::W == 128) return (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  return (c >> 2) * 1024 + r * 64 + (((c & 3) ^ ((r >> 1) & 3)) << 4);
}

// Key of index g within eight: 0 5 2 7 4 1 6 3.  A K load's phase takes keys
// key_of(2p), key_of(2p + 1) at pieces t (mod 4), a V load's the keys
// key_of(2t) or key_of(2t + 1) at pieces 2p, 2p + 1 (t = 0..3): the first two
// differ in bit 2, the other four in bits 1 and 2, so the swizzle sends the
// eight pieces to different banks.
__device__ __forceinline__ int key_of(int g) { return g ^ ((g & 1) << 2); }

template <typename T> __device__ __forceinline__ float2 up2(uint32_t x);
template <> __device__ __forceinline__ float2 up2<__nv_bfloat16>(uint32_t x) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x));
}
template <> __device__ __forceinline__ float2 up2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T> __device__ __forceinline__ uint32_t pack_t2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack_t2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack_t2<__half>(float a, float b) { return pack_h2(a, b); }

// Two columns of a finished row: O / l, and with the first ones the LSE.
template <typename T>
__device__ __forceinline__ void store_pair(const Args& A, const Job& J, int hk, int row, int c, float x, float y, float top,
                                           float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int tk = (J.row0 + row) / A.g, h = hk * A.g + J.row0 + row - tk * A.g;
  T* dst = static_cast<T*>(A.o) + elem_off(A.so, (long long)J.q0 + tk, h) + c;
  *reinterpret_cast<uint32_t*>(dst) = pack_t2<T>(x * inv, y * inv);
  if (c == 0)
    A.lse[(long long)h * A.total_q + J.q0 + tk] =
        l == 0.f ? -INFINITY : (top - P_LOG2 + log2f(l)) * 0.6931471805599453f;
}

// Four of them.
template <typename T>
__device__ __forceinline__ void store_row(const Args& A, const Job& J, int hk, int row, int c, const float4& v, float top,
                                          float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int tk = (J.row0 + row) / A.g, h = hk * A.g + J.row0 + row - tk * A.g;
  T* dst = static_cast<T*>(A.o) + elem_off(A.so, (long long)J.q0 + tk, h) + c;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_t2<T>(v.x * inv, v.y * inv), pack_t2<T>(v.z * inv, v.w * inv));
  if (c == 0)
    A.lse[(long long)h * A.total_q + J.q0 + tk] =
        l == 0.f ? -INFINITY : (top - P_LOG2 + log2f(l)) * 0.6931471805599453f;
}

// An 8 x 8 matrix of 16-bit values, a row over four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int DQK, int DV, int NT, typename T>
__global__ void __launch_bounds__(NTHREADS, Cfg<DQK, DV, NT>::RESIDENT) kv_fwd_kernel(const __grid_constant__ Maps maps, const Args A) {
  using C = Cfg<DQK, DV, NT>;
  constexpr int ROWS = C::ROWS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);   // the swizzle counts from 1024
  int2* meta = reinterpret_cast<int2*>(smem + C::OFF_META);
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* s_l = s_m + NWARPS * ROWS;
  float2* s_jml = reinterpret_cast<float2*>(s_l + NWARPS * ROWS);   // [ROWS]
  int* s_bad = reinterpret_cast<int*>(s_jml + ROWS);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

  // block -> (slot, kv head, split) -> (request, row tile)
  const int job = blockIdx.x / A.nsplit, split = blockIdx.x - job * A.nsplit;
  const int slot = job / A.c.hkv, hk = job - slot * A.c.hkv;
  const Slot at = slot_of<ROWS>(A, slot);
  const int b = at.b;
  MaskArgs mk;
  Job J = make_job<ROWS>(A, b, at.m, mk);
  if (split == 0 && hk == 0 && misses<ROWS>(A, slot)) J.bad = true;   // reported
  const int per_split = split_tiles(A, J);
  const bool whole = J.ntile <= per_split;        // no other split holds keys of these rows
  const int tile0 = split * per_split;
  if (J.nrow <= 0 || (split > 0 && tile0 >= J.ntile)) {
    if (tid == 0) A.status[blockIdx.x] = J.bad ? ATTN_ERR_BAD_SEQLENS : ATTN_OK;
    // a cluster whose rows have splits to join (the same for all of it) meets twice
    if (A.cluster && J.nrow > 0 && !whole) {
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * C::NST;
  if (tid == 0) *s_bad = 0;
  if (lane == 0) {
    for (int i = 0; i < C::NST; ++i) ptx::mbar_init(bars + i, 1);
    ptx::fence_mbar_init();
  }
  const int ntile = min(per_split, J.ntile - tile0);      // may be <= 0 for split 0
  const int key0 = J.kbeg + tile0 * TILE;
  const int shift = A.c.page_shift, in_page = (1 << shift) - 1;
  const int page0 = key0 >> shift;
  const int* table = A.table + b * A.table_stride + page0;
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::RING;
  int at_in = 0, at_out = 0;      // stages of the ring to fill and to read next, the latter's phase
  uint32_t parity = 0;
  auto advance = [&](int at) { return at + 1 == C::NST ? 0 : at + 1; };
  // tile i of the split, of this page, into the next stage (lane 0): every tile
  // completes its barrier once
  auto load = [&](int i, int page) {
    const int row = (key0 + i * TILE) & in_page;
    const uint32_t st = ring + at_in * C::STAGE;
    if (page >= 0 && page < A.c.num_pages) {
      ptx::mbar_arrive_expect_tx(bars + at_in, C::STAGE);
#pragma unroll
      for (int c = 0; c < Box<DQK>::N; ++c)
        tma_load_4d(st + c * TILE * Box<DQK>::W, &maps.k, bars + at_in, c * Box<DQK>::W, hk, row, page);
#pragma unroll
      for (int c = 0; c < Box<DV>::N; ++c)
        tma_load_4d(st + C::KB + c * TILE * Box<DV>::W, &maps.v, bars + at_in, c * Box<DV>::W, hk, row, page);
    } else {
      ptx::mbar_arrive(bars + at_in);
    }
  };
  // tiles [from, to) are worked on with their pages in shared memory; the first
  // ones leave before anything else is known
  auto start = [&](int from, int to) {
    int first[C::NST - 1];
#pragma unroll
    for (int s = 0; s < C::NST - 1; ++s) {
      const int i = from + warp + s * NWARPS;
      first[s] = lane == 0 && i < to ? __ldg(table + (((key0 + i * TILE) >> shift) - page0)) : -1;
    }
#pragma unroll
    for (int s = 0; s < C::NST - 1; ++s) {
      const int i = from + warp + s * NWARPS;
      if (i < to) {
        if (lane == 0) load(i, first[s]);
        at_in = advance(at_in);
      }
    }
  };
  start(0, min(ntile, META_TILES));

  // row g of each row group of q, as fp16 under a power of two; a negative
  // softmax scale goes into its sign, so scores and their factors order alike
  uint32_t qb[NT][DQK / 16][2];
  float rs[NT][2];                       // log2 units per raw score of rows 2t, 2t + 1
  int tok[NT][2];
  const float sign = A.scale_log2 < 0.f ? -1.f : 1.f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = min(J.row0 + 8 * n + g, J.row0 + J.nrow - 1);   // rows past the end repeat the last
    const int i = row / A.g;
    const T* qp = static_cast<const T*>(A.q) + elem_off(A.sq, (long long)J.q0 + i, hk * A.g + row - i * A.g);
    uint4 raw[DQK / 32];
    float mx = 0.f;
#pragma unroll
    for (int c = 0; c < DQK / 64; ++c) {
      const uint4* p = reinterpret_cast<const uint4*>(qp + (t + 4 * c) * 16);
      raw[2 * c] = __ldg(p);
      raw[2 * c + 1] = __ldg(p + 1);
    }
#pragma unroll
    for (int i = 0; i < DQK / 32; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
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
    const float up = sign * exp2_int(14 - e);
    const float unit = fabsf(A.scale_log2) * exp2_int(e - 14);
#pragma unroll
    for (int i = 0; i < DQK / 32; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {        // 16 elements in two pieces: k-step 4 (i / 2) + 2 (i & 1) + k / 2
        const float2 f = up2<T>(w[k]);
        qb[n][(i >> 1) * 4 + (i & 1) * 2 + (k >> 1)][k & 1] = pack_h2(f.x * up, f.y * up);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {          // row 2t + r is lane group 2t + r's
      rs[n][r] = __shfl_sync(0xffffffffu, unit, (2 * t + r) * 4);
      tok[n][r] = min(J.row0 + 8 * n + 2 * t + r, J.row0 + J.nrow - 1) / A.g;
    }
  }

  constexpr int MT = DV / 16;     // tiles of 16 value columns
  float o[NT][MT][4];
  float mrow[NT][2], lrow[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[n][j][k] = 0.f;
    mrow[n][0] = mrow[n][1] = -INFINITY;
    lrow[n][0] = lrow[n][1] = 0.f;
  }
  int unit = 0;                   // the accumulator counts in 2^unit
  const int itok0 = J.row0 / A.g, itok1 = (J.row0 + J.nrow - 1) / A.g;

  bool arrived = true;
  for (int from = 0; from < ntile; from += META_TILES) {
    const int to = min(ntile, from + META_TILES), meta0 = (key0 + from * TILE) >> shift;
    if (from > 0 && arrived) start(from, to);
    __syncthreads();   // the pages before these have been used
    for (int i = tid; i <= ((key0 + to * TILE - 1) >> shift) - meta0; i += NTHREADS) {
      const int page = __ldg(table + (meta0 - page0) + i);
      if (page >= 0 && page < A.c.num_pages) {
        const long long at = (long long)page * A.c.hkv + hk;
        const int ek = kv_exp_of(__ldg(A.c.k_exp + at)), ev = kv_exp_of(__ldg(A.c.v_exp + at));
        meta[i] = make_int2(page, (ek & 0xffff) | (ev << 16));
      } else {
        *s_bad = 1;
        meta[i] = make_int2(-1, 0);
      }
    }
    __syncthreads();
    for (int i = from + warp; arrived && i < to; i += NWARPS) {
      const int ahead = i + (C::NST - 1) * NWARPS;
      if (ahead < to) {
        if (lane == 0) load(ahead, meta[((key0 + ahead * TILE) >> shift) - meta0].x);
        at_in = advance(at_in);
      }
      const int key = key0 + i * TILE;
      const int2 mt = meta[(key >> shift) - meta0];
      const uint32_t st = ring + at_out * C::STAGE;
      arrived = __all_sync(0xffffffffu, wait_bar(ptx::smem_u32(bars + at_out), parity));
      if (!arrived) {
        // give the copies still in flight as long again before the memory is used
        for (int j = 0; j < C::NST && i + j * NWARPS < to; ++j) {
          wait_bar(ptx::smem_u32(bars + at_out), parity);
          at_out = advance(at_out);
          parity ^= at_out == 0;
        }
        break;
      }
      at_out = advance(at_out);
      parity ^= at_out == 0;
      if (mt.x >= 0) {
        const bool inside = key >= J.klo && key + TILE - 1 <= J.khi;
        if (!inside) {
          // rows that no query sees may hold anything: zero V there (masked
          // scores make their weights 0, but 0 NaN is NaN)
          for (int n = lane; n < TILE * (DV / 16); n += 32) {
            const int r = n / (DV / 16), c = n % (DV / 16);
            if (key + r < J.klo || key + r > J.khi)
              *reinterpret_cast<uint4*>(smem + warp * C::RING + (st - ring) + C::KB + off<DV>(r, c)) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();   // before the stage is refilled by TMA
          __syncwarp();
        }
        // S^T = K Q^T: keys key_of(g) and 8 more, rows 2t and 2t + 1
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[n][k] = 0.f;
#pragma unroll
        for (int c = 0; c < DQK / 64; ++c) {
          const uint4 w0 = lds128(st + off<DQK>(key_of(g), t + 4 * c)), w1 = lds128(st + off<DQK>(8 + key_of(g), t + 4 * c));
          const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a[4] = {e4m3x2_to_h2((uint16_t)a0[k]), e4m3x2_to_h2((uint16_t)a1[k]),
                                   e4m3x2_to_h2((uint16_t)(a0[k] >> 16)), e4m3x2_to_h2((uint16_t)(a1[k] >> 16))};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[n], a, qb[n][4 * c + k][0], qb[n][4 * c + k][1]);
          }
        }
        const float ks = exp2_int((int)(short)(mt.y & 0xffff));
        const bool full = inside &&
                          (mk.right < 0 || key + TILE - 1 <= (long long)itok0 + mk.off + mk.right) &&
                          (mk.left < 0 || key >= (long long)itok1 + mk.off - mk.left);
        if (!full) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int kk = key + key_of(g) + 8 * (k >> 1);
              if (kk < J.klo || kk > J.khi || !sees(mk, tok[n][k & 1], kk)) s[n][k] = -INFINITY;
            }
        }
        bool grow = false;
        float f[NT][2], top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            f[n][r] = fmaxf(rs[n][r] * ks, 1.17549435e-38f);   // never 0: a masked score stays -inf
            top[n][r] = fmaxf(s[n][r], s[n][2 + r]) * f[n][r];
            grow |= top[n][r] > mrow[n][r] + SLACK_LOG2;
          }
        const int ev = mt.y >> 16;
        grow = __any_sync(0xffffffffu, grow);
        if (grow || ev > unit + EV_SLACK || ev < unit - EV_SLACK) {
          const float de = exp2_int(unit - ev);
          unit = ev;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float a[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float x = top[n][r];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              a[r] = 1.f;
              if (x > mrow[n][r]) {
                a[r] = fast_exp2(mrow[n][r] - x);   // 0 from -inf
                mrow[n][r] = x;
              }
              lrow[n][r] *= a[r];
              a[r] *= de;
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[n][j][k] *= a[k & 1];
          }
        }
        const float ratio = exp2_int(ev - unit);
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float r0 = mrow[n][0] == -INFINITY ? 0.f : P_LOG2 - mrow[n][0];
          const float r1 = mrow[n][1] == -INFINITY ? 0.f : P_LOG2 - mrow[n][1];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float p0 = fast_exp2(fmaf(s[n][2 * j], f[n][0], r0)), p1 = fast_exp2(fmaf(s[n][2 * j + 1], f[n][1], r1));
            lrow[n][0] += p0;
            lrow[n][1] += p1;
            pb[n][j] = transpose8x8(pack_h2(p0 * ratio, p1 * ratio));
          }
        }
        // O^T += V^T P^T: keys key_of(2t), key_of(2t + 1) and 8 more are this lane's
        // rows of V; column tile j holds elements 2j (its rows 0-7) and 2j + 1 of each lane
        // group's consecutive columns
        const uint32_t vt = st + C::KB;
        auto columns = [&](int j, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
          const uint32_t lo0 = __byte_perm(w0, w1, 0x5140), hi0 = __byte_perm(w0, w1, 0x7362);
          const uint32_t lo1 = __byte_perm(w2, w3, 0x5140), hi1 = __byte_perm(w2, w3, 0x7362);
          const uint32_t a[4] = {e4m3x2_to_h2((uint16_t)lo0), e4m3x2_to_h2((uint16_t)(lo0 >> 16)),
                                 e4m3x2_to_h2((uint16_t)lo1), e4m3x2_to_h2((uint16_t)(lo1 >> 16))};
          const uint32_t c[4] = {e4m3x2_to_h2((uint16_t)hi0), e4m3x2_to_h2((uint16_t)(hi0 >> 16)),
                                 e4m3x2_to_h2((uint16_t)hi1), e4m3x2_to_h2((uint16_t)(hi1 >> 16))};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(o[n][j], a, pb[n][0], pb[n][1]);
            mma16816(o[n][j + 1], c, pb[n][0], pb[n][1]);
          }
        };
        const int v0 = key_of(2 * t), v1 = key_of(2 * t + 1);
        if (DV == 64) {
          const int c = g >> 1, h8 = (g & 1) * 8;
          const uint2 w0 = lds64(vt + off<DV>(v0, c) + h8), w1 = lds64(vt + off<DV>(v1, c) + h8);
          const uint2 w2 = lds64(vt + off<DV>(v0 + 8, c) + h8), w3 = lds64(vt + off<DV>(v1 + 8, c) + h8);
          columns(0, w0.x, w1.x, w2.x, w3.x);
          columns(2, w0.y, w1.y, w2.y, w3.y);
        } else {
#pragma unroll
          for (int half = 0; half < DV / 128; ++half) {
            const int c = g + 8 * half;
            const uint4 w0 = lds128(vt + off<DV>(v0, c)), w1 = lds128(vt + off<DV>(v1, c));
            const uint4 w2 = lds128(vt + off<DV>(v0 + 8, c)), w3 = lds128(vt + off<DV>(v1 + 8, c));
            columns(8 * half, w0.x, w1.x, w2.x, w3.x);
            columns(8 * half + 2, w0.y, w1.y, w2.y, w3.y);
            columns(8 * half + 4, w0.z, w1.z, w2.z, w3.z);
            columns(8 * half + 6, w0.w, w1.w, w2.w, w3.w);
          }
        }
      }
      __syncwarp();   // the stage may be refilled
    }
  }
  if (!arrived) {   // a load did not arrive: no result instead of a wrong one
    *s_bad = 2;
#pragma unroll
    for (int n = 0; n < NT; ++n) lrow[n][0] = lrow[n][1] = __int_as_float(0x7fc00000);
  }

  // join the warps: maxima and sums, then each warp's O under the common maximum
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float l = lrow[n][r];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {
        s_m[warp * ROWS + 8 * n + 2 * t + r] = mrow[n][r];
        s_l[warp * ROWS + 8 * n + 2 * t + r] = l;
      }
    }
  __syncthreads();   // also: every ring has been read
  float* so = reinterpret_cast<float*>(smem);   // [NWARPS][ROWS][DV]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * n + 2 * t + r;
      float top = s_m[row];
#pragma unroll
      for (int w = 1; w < NWARPS; ++w) top = fmaxf(top, s_m[w * ROWS + row]);
      // a warp that saw no key of the row holds zeros (or NaN, which stays)
      const float a = (mrow[n][r] == -INFINITY ? 1.f : fast_exp2(mrow[n][r] - top)) * exp2_int(unit);
      float* dst = so + (warp * ROWS + row) * DV;
      constexpr int RUN = DV == 64 ? 8 : 16;    // consecutive columns of a lane group
#pragma unroll
      for (int j = 0; j < MT; j += 2)
        *reinterpret_cast<float4*>(dst + (2 * j / RUN) * 128 + g * RUN + 2 * j % RUN) =
            make_float4(o[n][j][r] * a, o[n][j][2 + r] * a, o[n][j + 1][r] * a, o[n][j + 1][2 + r] * a);
    }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long part = blockIdx.x;
  float* s_join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
  const int pieces = J.nrow * (DV / 4);
  for (int i = tid; i < pieces; i += NTHREADS) {
    const int row = i / (DV / 4), c = (i % (DV / 4)) * 4;
    float top = s_m[row];
#pragma unroll
    for (int w = 1; w < NWARPS; ++w) top = fmaxf(top, s_m[w * ROWS + row]);
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
      const float mw = s_m[w * ROWS + row], lw = s_l[w * ROWS + row];
      l += mw == -INFINITY ? lw : lw * fast_exp2(mw - top);   // lw is 0 there, or NaN
      const float4 y = *reinterpret_cast<const float4*>(so + (w * ROWS + row) * DV + c);
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    if (whole) {
      store_row<T>(A, J, hk, row, c, v, top, l);
    } else if (A.cluster) {
      *reinterpret_cast<float4*>(s_join + row * DV + c) = v;
      if (c == 0) s_jml[row] = make_float2(top, l);
    } else {
      *reinterpret_cast<float4*>(A.part_o + (part * A.job_rows + row) * DV + c) = v;
      if (c == 0) A.part_ml[part * A.job_rows + row] = make_float2(top, l);
    }
  }
  if (A.cluster && !whole) {
    // each CTA finishes its share of the rows' pieces
    cluster_arrive();
    cluster_wait();
    const int n = cdiv(J.ntile, per_split);
    const uint32_t join = ptx::smem_u32(s_join), jml = ptx::smem_u32(s_jml);
    for (int i = split * NTHREADS + tid; i < pieces; i += n * NTHREADS) {
      const int row = i / (DV / 4), c = (i % (DV / 4)) * 4;
      float tops[MAX_CLUSTER], top = -INFINITY;
#pragma unroll
      for (int s = 0; s < MAX_CLUSTER; ++s) {
        tops[s] = s < n ? ld_cluster(in_cta(jml + row * 8, s)) : -INFINITY;
        top = fmaxf(top, tops[s]);
      }
      float l = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < MAX_CLUSTER; ++s) {
        if (s >= n) break;
        const float ls = ld_cluster(in_cta(jml + row * 8 + 4, s));
        const float4 y = ld_cluster4(in_cta(join + (row * DV + c) * 4, s));
        // a split that saw no key of the row holds zeros (or NaN, which stays)
        const float w = tops[s] == -INFINITY ? 1.f : fast_exp2(tops[s] - top);
        l += w * ls;
        v.x += w * y.x; v.y += w * y.y; v.z += w * y.z; v.w += w * y.w;
      }
      store_row<T>(A, J, hk, row, c, v, top, l);
    }
    cluster_arrive();   // no CTA leaves while its memory is read
    cluster_wait();
  }
  if (tid == 0)
    A.status[blockIdx.x] = *s_bad == 2 ? ATTN_ERR_TIMEOUT
                           : J.bad     ? ATTN_ERR_BAD_SEQLENS
                           : *s_bad    ? ATTN_ERR_BAD_PAGE
                                       : ATTN_OK;
}

// The joins: O = sum 2^(m_s - m) O_s / sum 2^(m_s - m) l_s over a row's splits, in
// a fixed order.  A split that saw no key of the row holds zeros (or NaN, which
// stays).
//
// Many rows of few splits: a warp takes a row, DV / 32 columns to a lane.  Rows
// with nothing to join cost their lengths' loads (512 jobs of 4 rows: 2 us less
// than a CTA to each row).
template <int DV, int NT, typename T>
__global__ void __launch_bounds__(NTHREADS) join_rows_kernel(const Args A, long long rows) {
  constexpr int ROWS = 8 * NT, PER = DV / 32 >= 4 ? 4 : 2, REPS = DV / 32 / PER;   // columns in runs of PER
  const int lane = threadIdx.x & 31;
  long long x = (long long)blockIdx.x * NWARPS + (threadIdx.x >> 5);
  const bool some = x < rows;
  if (!some) x = 0;
  const int row = (int)(x % A.job_rows);
  const long long job = x / A.job_rows;
  const int slot = (int)(job / A.c.hkv), hk = (int)(job - (long long)slot * A.c.hkv);
  const Slot at = slot_of<ROWS>(A, slot);
  MaskArgs mk;
  const Job J = make_job<ROWS>(A, at.b, at.m, mk);
  const int n = cdiv(J.ntile, split_tiles(A, J));
  // launched early: the splits' kernel ends here.  Every thread waits, also where
  // nothing is to join: what follows on the stream waits for this kernel alone.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!some || row >= J.nrow || n <= 1) return;
  const float2* ml = A.part_ml + job * A.nsplit * A.job_rows + row;
  const float* po = A.part_o + (job * A.nsplit * A.job_rows + row) * DV + lane * PER;
  float top = -INFINITY;
  for (int s = lane; s < n; s += 32) top = fmaxf(top, ml[s * A.job_rows].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float l = 0.f, v[REPS][PER];
#pragma unroll
  for (int r = 0; r < REPS; ++r)
#pragma unroll
    for (int k = 0; k < PER; ++k) v[r][k] = 0.f;
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float2 y = ml[s * A.job_rows];
    const float w = y.x == -INFINITY ? 1.f : fast_exp2(y.x - top);
    l += w * y.y;
    const float* src = po + (long long)s * A.job_rows * DV;
#pragma unroll
    for (int r = 0; r < REPS; ++r)
#pragma unroll
      for (int k = 0; k < PER; k += 2) {
        const float2 z = *reinterpret_cast<const float2*>(src + r * 32 * PER + k);
        v[r][k] += w * z.x;
        v[r][k + 1] += w * z.y;
      }
  }
#pragma unroll
  for (int r = 0; r < REPS; ++r)
#pragma unroll
    for (int k = 0; k < PER; k += 2) store_pair<T>(A, J, hk, row, r * 32 * PER + lane * PER + k, v[r][k], v[r][k + 1], top, l);
}

// Few rows of many splits: a CTA takes a row; DV / 4 threads cover its columns, and
// the thread groups take the splits in turn: blockDim.x follows their number.
constexpr int JOIN_THREADS = 512;   // at most

template <int DV, int NT, typename T>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const Args A) {
  constexpr int ROWS = 8 * NT;
  constexpr int COLS = DV / 4;
  __shared__ float4 s_v[JOIN_THREADS / COLS][COLS];
  __shared__ float s_l[JOIN_THREADS / COLS];
  __shared__ float s_top[JOIN_THREADS / 32];
  const int groups = blockDim.x / COLS, nw = blockDim.x / 32;
  const int job = blockIdx.x / A.job_rows, row = blockIdx.x % A.job_rows;
  const int grp = threadIdx.x / COLS, col = threadIdx.x % COLS, c = col * 4;
  const int slot = job / A.c.hkv, hk = job - slot * A.c.hkv;
  const Slot at = slot_of<ROWS>(A, slot);
  MaskArgs mk;
  const Job J = make_job<ROWS>(A, at.b, at.m, mk);
  const int n = cdiv(J.ntile, split_tiles(A, J));
  asm volatile("griddepcontrol.wait;" ::: "memory");   // all threads: see join_rows_kernel
  if (row >= J.nrow || n <= 1) return;
  const float2* ml = A.part_ml + (long long)job * A.nsplit * A.job_rows + row;
  const float* po = A.part_o + ((long long)job * A.nsplit * A.job_rows + row) * DV + c;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < n; s += blockDim.x) top = fmaxf(top, ml[s * A.job_rows].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < nw; ++w) top = fmaxf(top, s_top[w]);
  float l = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = grp; s < n; s += groups) {
    const float2 x = ml[s * A.job_rows];
    const float4 y = *reinterpret_cast<const float4*>(po + (long long)s * A.job_rows * DV);
    // a split that saw no key of the row holds zeros (or NaN, which stays)
    const float w = x.x == -INFINITY ? 1.f : fast_exp2(x.x - top);
    l += w * x.y;
    v.x += w * y.x; v.y += w * y.y; v.z += w * y.z; v.w += w * y.w;
  }
  s_v[grp][col] = v;
  if (col == 0) s_l[grp] = l;
  __syncthreads();
  if (grp == 0) {
    const int used = min(groups, n);
    for (int w = 1; w < used; ++w) {
      const float4 y = s_v[w][col];
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
      l += s_l[w];
    }
    store_row<T>(A, J, hk, row, c, v, top, l);
  }
}

// ---------------------------------------------------------------- host side

struct Layout {
  int nt, mtiles, job_rows, nsplit, min_tiles;
  long long jobs;
  bool cluster, direct;
  size_t off_status, off_ml, off_o, off_long, total;
  KvLong lng;
};

static int max_keys(const attn_kv_fwd_params& p) {
  const long long cap = (long long)p.max_blocks * p.cache.page_size;
  return (int)(cap < p.max_seqlen_k ? cap : p.max_seqlen_k);
}

static Layout layout(const attn_kv_fwd_params& p) {
  Layout L{};
  const int g = p.nhead_q / p.cache.nhead_kv;
  L.lng = kv_long_layout(p, max_keys(p));
  int most = p.max_seqlen_q < L.lng.from ? p.max_seqlen_q : L.lng.from;   // query tokens of this path
  most = most < p.total_q ? most : p.total_q;
  const long long rows = (long long)(most > 0 ? most : 1) * g, all_rows = (long long)p.total_q * g;
  // tiles of 8 rows where a request has no more, at least on average
  L.nt = rows <= 8 || all_rows <= 8LL * p.batch ? 1 : 2;
  L.mtiles = (int)cdiv_ll(rows, 8 * L.nt);
  L.job_rows = (int)(rows < 8 * L.nt ? rows : 8 * L.nt);
  const long long packed = all_rows / (8 * L.nt) + p.batch, each = (long long)p.batch * L.mtiles;
  L.direct = each <= packed;
  L.jobs = p.cache.nhead_kv * (L.direct ? each : packed);
  // Keys that the rows of a job see at most (8 requests of up to 1,183 tokens under
  // a window of 190, head dim 256: 8.8 us, 18.1 with splits for all of them).
  long long keys = max_keys(p);
  if (p.mask == ATTN_MASK_WINDOW && p.window_left >= 0 && p.window_right >= 0) {
    const long long span = (long long)p.window_left + p.window_right + 1 + cdiv(8 * L.nt, g);
    keys = span < keys ? span : keys;
  }
  const int tiles = (int)(keys / TILE) + 2;
  const int wave = SMS * resident(p.cache.d_qk, L.nt);
  const bool few = 2 * L.jobs <= wave;
  L.min_tiles = few ? MIN_TILES : EVEN_TILES;
  const long long n = few ? (p.batch > 1 ? wave : HALF_WAVE) / L.jobs : cdiv_ll(MAX_GRID, L.jobs);
  L.nsplit = n < cdiv(tiles, L.min_tiles) ? (int)n : cdiv(tiles, L.min_tiles);
  // clusters of one wave: a cluster stays within eighteen SMs or so
  L.cluster = few && L.nsplit > 1 && L.nsplit <= MAX_CLUSTER && L.jobs <= 8 * (wave * 18 / SMS / L.nsplit);
  auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  size_t o = 0;
  L.off_status = o;
  o = up(o + (size_t)L.jobs * L.nsplit * sizeof(int));
  const size_t parts = L.nsplit > 1 && !L.cluster ? (size_t)L.jobs * L.nsplit : 0;
  L.off_ml = o;
  o = up(o + parts * L.job_rows * sizeof(float2));
  L.off_o = o;
  o = up(o + parts * L.job_rows * p.cache.d_v * sizeof(float));
  L.off_long = o;
  L.total = o + L.lng.total;
  return L;
}

// The checks that need no pointers (the sizing call's).
static int validate_sizes(const attn_kv_fwd_params* p) {
  if (!p || p->reserved != 0 || (p->dtype != ATTN_BF16 && p->dtype != ATTN_FP16)) return ATTN_ERR_INVALID_ARG;
  const attn_kv_cache& c = p->cache;
  if (c.num_pages < 1 || c.nhead_kv < 1 || c.nhead_kv > KV_MAX_HEADS || c.reserved != 0 || kv_page_shift(c.page_size) < 0)
    return ATTN_ERR_INVALID_ARG;
  if (!kv_headdims(c.d_qk, c.d_v)) return ATTN_ERR_UNSUPPORTED_HEADDIM;
  if (p->batch < 1 || p->batch > (1 << 20) || p->nhead_q < 1 || p->nhead_q > (1 << 16) || p->nhead_q % c.nhead_kv)
    return ATTN_ERR_INVALID_ARG;
  if (p->total_q < 0 || p->total_q > (1 << 30) || p->max_seqlen_q < 0 || p->max_seqlen_q > (1 << 30) ||
      p->max_seqlen_k < 0 || p->max_seqlen_k > (1 << 30) || p->max_blocks < 1 ||
      (long long)p->max_blocks * c.page_size > (1LL << 30))
    return ATTN_ERR_INVALID_ARG;
  if (p->mask < ATTN_MASK_NONE || p->mask > ATTN_MASK_WINDOW) return ATTN_ERR_INVALID_ARG;
  if (p->mask == ATTN_MASK_WINDOW && (p->window_left < -1 || p->window_right < -1)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->softmax_scale) || p->softmax_scale == 0.f) return ATTN_ERR_INVALID_ARG;
  // rows of a group and the grid fit 32 bits
  const long long rows = (long long)p->max_seqlen_q * (p->nhead_q / c.nhead_kv);
  if (rows > (1LL << 30)) return ATTN_ERR_INVALID_ARG;
  const Layout L = layout(*p);
  if (L.jobs * L.nsplit > (1LL << 30) || L.jobs > (1LL << 26)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

// The cache as (d, heads, rows of a page, pages), boxes of one head's 16 rows.
template <int D>
static bool make_map(CUtensorMap* m, const void* base, const KvCacheView& c, const KvStrides& s) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {D, (cuuint64_t)c.hkv, (cuuint64_t)1 << c.page_shift, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)s.h, (cuuint64_t)s.r, (cuuint64_t)s.p};
  const cuuint32_t box[4] = {Box<D>::W, 1, TILE, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, Box<D>::W == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DQK, int DV, int NT, typename T>
static int launch(const Args& a, long long jobs, cudaStream_t st) {
  using C = Cfg<DQK, DV, NT>;
  Maps maps;
  if (!make_map<DQK>(&maps.k, a.c.k, a.c, a.c.sk) || !make_map<DV>(&maps.v, a.c.v, a.c, a.c.sv)) return ATTN_ERR_CUDA;
  auto kern = kv_fwd_kernel<DQK, DV, NT, T>;
  if (!succeeded(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)))
    return ATTN_ERR_CUDA;
  if (a.cluster) {
    cudaLaunchAttribute dims;
    dims.id = cudaLaunchAttributeClusterDimension;
    dims.val.clusterDim.x = a.nsplit;
    dims.val.clusterDim.y = dims.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(jobs * a.nsplit));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = &dims;
    cfg.numAttrs = 1;
    return succeeded(cudaLaunchKernelEx(&cfg, kern, maps, a)) ? ATTN_OK : ATTN_ERR_CUDA;
  }
  kern<<<(unsigned)(jobs * a.nsplit), NTHREADS, C::SMEM, st>>>(maps, a);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;   // no parts to join
  if (a.nsplit > 1) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const long long rows = jobs * a.job_rows;
    if (jobs >= HALF_WAVE) {
      cfg.gridDim = dim3((unsigned)cdiv_ll(rows, NWARPS));
      cfg.blockDim = dim3(NTHREADS);
      if (!succeeded(cudaLaunchKernelEx(&cfg, join_rows_kernel<DV, NT, T>, a, rows))) return ATTN_ERR_CUDA;
    } else {
      int threads = NTHREADS;   // about four splits to a thread group
      while (threads < JOIN_THREADS && threads / (DV / 4) * 4 < a.nsplit) threads *= 2;
      cfg.gridDim = dim3((unsigned)rows);
      cfg.blockDim = dim3(threads);
      if (!succeeded(cudaLaunchKernelEx(&cfg, join_kernel<DV, NT, T>, a))) return ATTN_ERR_CUDA;
    }
  }
  return ATTN_OK;
}

template <int DQK, int DV, typename T>
static int launch_rows(const Args& a, const Layout& L, cudaStream_t st) {
  return L.nt == 1 ? launch<DQK, DV, 1, T>(a, L.jobs, st) : launch<DQK, DV, 2, T>(a, L.jobs, st);
}

template <typename T>
static int launch_dims(const Args& a, const Layout& L, int dqk, int dv, cudaStream_t st) {
  if (dqk == 64) return launch_rows<64, 64, T>(a, L, st);
  if (dqk == 128) return launch_rows<128, 128, T>(a, L, st);
  if (dqk == 192) return launch_rows<192, 128, T>(a, L, st);
  return launch_rows<256, 256, T>(a, L, st);
}

static int run(const attn_kv_fwd_params* p, void* ws, size_t ws_bytes, cudaStream_t st) {
  int s = validate_sizes(p);
  if (s != ATTN_OK) return s;
  Args a{};
  if ((s = kv_resolve(p->cache, &a.c)) != ATTN_OK) return s;
  const int dqk = p->cache.d_qk, dv = p->cache.d_v;
  if (!packed_strides(p->stride_q, p->nhead_q, dqk, &a.sq) || !packed_strides(p->stride_o, p->nhead_q, dv, &a.so))
    return ATTN_ERR_INVALID_ARG;
  if (p->table_stride < p->max_blocks || p->table_stride >= (1LL << 36)) return ATTN_ERR_INVALID_ARG;
  const void* ints[] = {p->cu_seqlens_q, p->seqlens_k, p->block_table};
  for (const void* x : ints)
    if (!x || !aligned_to(x, 4)) return ATTN_ERR_INVALID_ARG;
  if (!aligned_to(p->cu_seqlens_q_padded, 4)) return ATTN_ERR_INVALID_ARG;
  const bool rows = p->total_q > 0;
  if ((rows && (!p->q || !p->o || !p->lse)) || !aligned_to(p->q, 16) || !aligned_to(p->o, 16) || !aligned_to(p->lse, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256)) return ATTN_ERR_INVALID_ARG;
  const Layout L = layout(*p);
  if (ws_bytes < L.total) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  char* w = static_cast<char*>(ws);
  a.q = p->q;
  a.o = p->o;
  a.lse = p->lse;
  a.cu_q = p->cu_seqlens_q;
  a.st_q = p->cu_seqlens_q_padded ? p->cu_seqlens_q_padded : p->cu_seqlens_q;
  a.len_k = p->seqlens_k;
  a.table = p->block_table;
  a.table_stride = p->table_stride;
  a.max_k = max_keys(*p);
  a.total_q = p->total_q;
  a.max_q = p->max_seqlen_q;
  a.batch = p->batch;
  a.hq = p->nhead_q;
  a.g = p->nhead_q / p->cache.nhead_kv;
  a.mask = p->mask;
  a.left = p->mask == ATTN_MASK_WINDOW ? p->window_left : -1;
  a.right = p->mask == ATTN_MASK_WINDOW ? p->window_right : -1;
  a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  a.nsplit = L.nsplit;
  a.min_tiles = L.min_tiles;
  a.cluster = L.cluster;
  a.direct = L.direct;
  a.mtiles = L.mtiles;
  a.long_from = L.lng.from;
  a.job_rows = L.job_rows;
  a.status = reinterpret_cast<int*>(w + L.off_status);
  a.part_ml = reinterpret_cast<float2*>(w + L.off_ml);
  a.part_o = reinterpret_cast<float*>(w + L.off_o);
  if (L.lng.slots > 0 && (s = launch_kv_long(*p, a.c, a.sq, a.so, a.max_k, L.lng, w + L.off_long, st)) != ATTN_OK) return s;
  if (p->dtype == ATTN_BF16) return launch_dims<__nv_bfloat16>(a, L, dqk, dv, st);
  return launch_dims<__half>(a, L, dqk, dv, st);
}

}  // namespace kvfwd
}  // namespace attn

using namespace attn;

extern "C" int attn_kv_fwd_workspace_size(const attn_kv_fwd_params* p, size_t* bytes) {
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  *bytes = 0;
  const int s = kvfwd::validate_sizes(p);
  if (s != ATTN_OK) return s;
  *bytes = kvfwd::layout(*p).total;
  return ATTN_OK;
}

extern "C" int attn_kv_fwd(const attn_kv_fwd_params* p, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return kvfwd::run(p, workspace, workspace_bytes, stream);
}

extern "C" int attn_kv_fwd_read_status(const attn_kv_fwd_params* p, const void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream, int* status) {
  if (!workspace || !status) return ATTN_ERR_INVALID_ARG;
  const int s = kvfwd::validate_sizes(p);
  if (s != ATTN_OK) return s;
  const kvfwd::Layout L = kvfwd::layout(*p);
  if (workspace_bytes < L.total) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  *status = ATTN_OK;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ATTN_ERR_CUDA;
  // in pieces that fit the stack (this library allocates nothing)
  int part[1024];
  const char* words[2] = {static_cast<const char*>(workspace) + L.off_status,
                          static_cast<const char*>(workspace) + L.off_long + kv_long_status_offset(L.lng)};
  const long long count[2] = {L.jobs * L.nsplit, L.lng.slots};
  for (int a = 0; a < 2; ++a)
    for (long long i = 0; i < count[a]; i += 1024) {
      const size_t k = (size_t)(count[a] - i < 1024 ? count[a] - i : 1024);
      if (cudaMemcpy(part, words[a] + i * sizeof(int), k * sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return ATTN_ERR_CUDA;
      for (size_t j = 0; j < k; ++j)
        if (part[j] != ATTN_OK && *status == ATTN_OK) *status = part[j];
    }
  return ATTN_OK;
}
