// Rotary positions of q and k (attn_rope): pair (a, b) of a row becomes
//   (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq.
//
// Memory bound: every element is read once and written once, the cosines are
// computed once per (row, pair) and shared by the row's heads through shared
// memory.
#include <cmath>

#include "common.cuh"
#include "kv_common.cuh"

namespace attn {
namespace rope {

constexpr int MAX_PAIRS = ATTN_ROPE_MAX_DIM / 2;
constexpr int NTHREADS = 256;
constexpr int RESIDENT = 5;   // CTAs per SM that the registers have to allow (58.7 us below; 62.3 with no bound, 62.6 at 6)

// Turns per position as a fraction of 2^64: position * step wraps exactly like
// the angle does, so no reduction error grows with the position.
struct Table {
  unsigned long long step[MAX_PAIRS];
  uint8_t axis[MAX_PAIRS];
};

struct Side {
  const void* in;
  void* out;
  long long ib, ir, ih, ob, orow, oh;   // element strides {batch, row, head}
};

struct Args {
  Side q, k;
  const int* pos;
  long long pa, pb, pr;
  int rows, seqlen, hq, heads, dim, half, inverse, tok;
};

// cos and sin of 2 pi x / 2^64.  The nearest quarter turn is split off in
// integers; the rest, at most an eighth of a turn, goes through the Taylor
// series of sine and cosine (remainders below (pi/4)^11 / 11! = 1.8e-9 and
// (pi/4)^12 / 12! = 1.2e-10).
__device__ __forceinline__ float2 cos_sin_turns(unsigned long long x) {
  const uint32_t u = (uint32_t)(x >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(u - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float z = r * r;
  float s = fmaf(z, 2.7557319224e-6f, -1.9841269841e-4f);
  s = fmaf(z, s, 8.3333333333e-3f);
  s = fmaf(z, s, -1.6666666667e-1f);
  s = fmaf(r * z, s, r);
  float c = fmaf(z, -2.7557319224e-7f, 2.4801587302e-5f);
  c = fmaf(z, c, -1.3888888889e-3f);
  c = fmaf(z, c, 4.1666666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  if (quarter & 1) {
    const float t = s;
    s = c;
    c = -t;
  }
  if (quarter & 2) {
    s = -s;
    c = -c;
  }
  return make_float2(c, s);
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// One chunk of a head's row: two vectors of VP elements.  Half split: VP
// elements of either rotated half, VP pairs; the columns past the rotated ones
// follow in chunks of two vectors that are copied.  Interleaved: 2 VP
// consecutive elements, pairs past the rotated ones copied.  VP = 8 (16-bit) or
// 4 (fp32) makes a vector one 16-byte access; VP = 1 takes fp32 rows of any
// alignment and size.  What else does not divide into such chunks is the staged
// kernel's below.
//
// A CTA takes `tok` rows; its threads walk over (row, head, chunk) in steps of
// NTHREADS.
template <typename T, int VP, bool INTER>
__global__ void __launch_bounds__(NTHREADS, RESIDENT) rope_kernel(const Args A, const __grid_constant__ Table table) {
  using V = Vec<T, VP>;
  extern __shared__ unsigned long long dyn[];
  unsigned long long* s_step = dyn;                                   // [half]
  float2* cs = reinterpret_cast<float2*>(dyn + cdiv(A.half, 2) * 2);  // [tok][chunks of pairs]
  int2* s_row = reinterpret_cast<int2*>(cs + A.tok * cdiv(A.half, VP) * VP);   // [tok]: batch entry, row
  uint8_t* s_axis = reinterpret_cast<uint8_t*>(s_row + A.tok);        // [half]
  // Pairs 2k and 2k + 1 of every chunk next to each other, then the next two of
  // every chunk: neighbouring threads (chunks) read neighbouring 16 bytes.
  const int full = (A.half + VP - 1) / VP;                            // chunks with a pair
  const int stride = full * VP;
  auto place = [&](int pair) {
    return VP == 1 ? pair : ((pair % VP / 2) * full + pair / VP) * 2 + pair % 2;
  };
  const int row0 = blockIdx.x * A.tok;
  const int nrow = min(A.tok, A.rows - row0);
  // the table comes from the parameter bank, which serves one address at a time
  for (int i = threadIdx.x; i < A.half; i += NTHREADS) {
    s_step[i] = table.step[i];
    s_axis[i] = table.axis[i];
  }
  if (threadIdx.x < nrow) {
    const int row = row0 + threadIdx.x, b = row / A.seqlen;
    s_row[threadIdx.x] = make_int2(b, row - b * A.seqlen);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nrow * A.half; i += NTHREADS) {
    const int rr = i / A.half, pair = i - rr * A.half;
    const int2 bs = s_row[rr];
    const int pos = __ldg(A.pos + s_axis[pair] * A.pa + bs.x * A.pb + bs.y * A.pr);
    float2 x = cos_sin_turns((unsigned long long)(long long)pos * s_step[pair]);
    if (A.inverse) x.y = -x.y;
    cs[rr * stride + place(pair)] = x;
  }
  __syncthreads();

  const int rot_chunks = INTER ? (A.dim + 2 * VP - 1) / (2 * VP) : A.half / VP;
  const int chunks = INTER ? rot_chunks : rot_chunks + (A.dim - 2 * A.half + 2 * VP - 1) / (2 * VP);
  // this thread's place among (row, head, chunk), and its step
  int c = threadIdx.x % chunks, h = threadIdx.x / chunks;
  int r = h / A.heads;
  h -= r * A.heads;
  const int dc = NTHREADS % chunks;
  int dh = NTHREADS / chunks;
  const int dr = dh / A.heads;
  dh -= dr * A.heads;
#pragma unroll 2
  while (r < nrow) {
    const bool turns = INTER || c < rot_chunks;
    const int at0 = INTER ? c * 2 * VP : turns ? c * VP : 2 * A.half + (c - rot_chunks) * 2 * VP;
    const int at1 = turns && !INTER ? at0 + A.half : at0 + VP;
    const int2 bs = s_row[r];
    const bool is_q = h < A.hq;
    const Side& x = is_q ? A.q : A.k;
    const int hh = is_q ? h : h - A.hq;
    const T* in = static_cast<const T*>(x.in) + bs.x * x.ib + bs.y * x.ir + hh * x.ih;
    T* out = static_cast<T*>(x.out) + bs.x * x.ob + bs.y * x.orow + hh * x.oh;
    V v0 = *reinterpret_cast<const V*>(in + at0), v1 = v0;
    if (at1 < A.dim) v1 = *reinterpret_cast<const V*>(in + at1);   // an odd last copy is one vector
    if (turns) {
      const float2* row_cs = cs + r * stride;
      float2 t[VP];
#pragma unroll
      for (int p = 0; p < VP; p += 2) {
        if (VP == 1) {
          t[0] = row_cs[INTER && c >= A.half ? 0 : c];
        } else {
          const float4 x = *reinterpret_cast<const float4*>(row_cs + ((p / 2) * full + (INTER && c >= full ? 0 : c)) * 2);
          t[p] = make_float2(x.x, x.y);
          t[p + 1 < VP ? p + 1 : p] = make_float2(x.z, x.w);
        }
      }
#pragma unroll
      for (int p = 0; p < VP; ++p) {
        if (INTER && c * VP + p >= A.half) break;   // copied
        // element of a and b of pair p among the 2 VP loaded ones
        const int ea = INTER ? 2 * p : p, eb = INTER ? 2 * p + 1 : p + VP;
        T& ra = ea < VP ? v0.v[ea] : v1.v[ea - VP];
        T& rb = eb < VP ? v0.v[eb] : v1.v[eb - VP];
        const float a = TypeOps<T>::to_f(ra), b = TypeOps<T>::to_f(rb);
        const float2 k = t[p];
        ra = TypeOps<T>::from_f(a * k.x - b * k.y);
        rb = TypeOps<T>::from_f(b * k.x + a * k.y);
      }
    }
    *reinterpret_cast<V*>(out + at0) = v0;
    if (at1 < A.dim) *reinterpret_cast<V*>(out + at1) = v1;
    c += dc;
    h += dh;
    r += dr;
    if (c >= chunks) {
      c -= chunks;
      ++h;
    }
    if (h >= A.heads) {
      h -= A.heads;
      ++r;
    }
  }
}

// Halves that start inside a 16-byte vector (half split, rot_dim no multiple of 16,
// or 8 for fp32), and interleaved rows that are an odd number of vectors.  A thread
// takes one vector of columns; a row's threads are in one warp, which passes the
// partners on through shared memory (five words per vector, nine cosines for eight:
// no bank conflicts), so rows still move in 16-byte pieces and may be rotated in
// place.  8,098 rows of 10 heads of 256, 250 rotated, fp16: 31.1 us, element by
// element 51.9.
template <typename T, bool INTER>
__global__ void __launch_bounds__(NTHREADS) rope_staged_kernel(const Args A, const __grid_constant__ Table table) {
  constexpr int E = 16 / sizeof(T);                      // elements of a vector
  constexpr int WARPS = NTHREADS / 32, MOST = ATTN_ROPE_MAX_DIM / E > 32 ? 2 : 1;   // vectors of a thread
  using V = Vec<T, E>;
  __shared__ uint32_t s_part[WARPS][32 * MOST * 5];
  __shared__ unsigned long long s_step[MAX_PAIRS];       // from the parameter bank, which serves one address at a time
  __shared__ uint8_t s_axis[MAX_PAIRS];
  extern __shared__ unsigned long long dyn[];
  float2* cs = reinterpret_cast<float2*>(dyn);
  const int stride = A.half + A.half / 8 + 1;
  if (threadIdx.x < A.half) {
    s_step[threadIdx.x] = table.step[threadIdx.x];
    s_axis[threadIdx.x] = table.axis[threadIdx.x];
  }
  __syncthreads();
  const int row0 = blockIdx.x * A.tok, nrow = min(A.tok, A.rows - row0);
  for (int i = threadIdx.x; i < nrow * A.half; i += NTHREADS) {
    const int rr = i / A.half, pair = i - rr * A.half, row = row0 + rr, b = row / A.seqlen;
    const int pos = __ldg(A.pos + s_axis[pair] * A.pa + b * A.pb + (row - b * A.seqlen) * A.pr);
    float2 x = cos_sin_turns((unsigned long long)(long long)pos * s_step[pair]);
    if (A.inverse) x.y = -x.y;
    cs[rr * stride + pair + pair / 8] = x;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vecs = A.dim / E, mine = cdiv(vecs, 32);     // vectors of a head's row, of a thread
  const int rows = mine > 1 ? 1 : 32 / vecs;             // heads' rows that a warp takes at a time
  const int sub = mine > 1 ? 0 : lane / vecs, c0 = mine > 1 ? lane : lane - sub * vecs;
  uint32_t* part = s_part[warp] + sub * vecs * 5;
  // a row's heads one after the other, its cosines in registers
  const int share = max(1, WARPS / nrow);                // warps of a row
  for (int r = warp / share; r < nrow; r += WARPS / share) {
    const int row = row0 + r, b = row / A.seqlen, s = row - b * A.seqlen;
    float2 t[MOST][E];                                   // cos, and sin as it multiplies the partner
#pragma unroll
    for (int k = 0; k < MOST; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int col = (c0 + 32 * k) * E + e;
        const bool first = INTER ? e % 2 == 0 : col < A.half;
        const int pair = min(INTER ? col / 2 : first ? col : col - A.half, A.half - 1);
        t[k][e] = cs[r * stride + pair + pair / 8];
        if (first) t[k][e].y = -t[k][e].y;
      }
    for (int h0 = warp % share * rows; h0 < A.heads; h0 += share * rows) {
      const int h = h0 + sub;
      const bool live = sub < rows && h < A.heads;
      const Side& x = h < A.hq ? A.q : A.k;
      const int hh = h < A.hq ? h : h - A.hq;
      const T* in = static_cast<const T*>(x.in) + b * x.ib + s * x.ir + hh * x.ih;
      T* out = static_cast<T*>(x.out) + b * x.ob + s * x.orow + hh * x.oh;
      V v[MOST];
#pragma unroll
      for (int k = 0; k < MOST; ++k) {
        const int c = c0 + 32 * k;
        if (!live || c >= vecs) continue;
        v[k] = *reinterpret_cast<const V*>(in + c * E);
        if (!INTER) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[k]);
#pragma unroll
          for (int i = 0; i < 4; ++i) part[c * 5 + i] = w[i];
        }
      }
      if (!INTER) __syncwarp();
#pragma unroll
      for (int k = 0; k < MOST; ++k) {
        const int c = c0 + 32 * k;
        if (!live || c >= vecs) continue;
        V y = v[k];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int col = c * E + e;
          const int other = col < A.half ? col + A.half : col - A.half;
          const float own = TypeOps<T>::to_f(v[k].v[e]);
          const float partner =
              TypeOps<T>::to_f(INTER ? v[k].v[e ^ 1] : reinterpret_cast<const T*>(part + other / E * 5)[other % E]);
          const T turned = TypeOps<T>::from_f(own * t[k][e].x + partner * t[k][e].y);
          if (col < 2 * A.half) y.v[e] = turned;         // the others are copied
        }
        *reinterpret_cast<V*>(out + c * E) = y;
      }
      if (!INTER) __syncwarp();                          // the parts may be overwritten
    }
  }
}

template <typename T>
static void launch_staged(const Args& a, const Table& t, bool inter, cudaStream_t st) {
  const int grid = cdiv(a.rows, a.tok);
  const size_t smem = (size_t)a.tok * (a.half + a.half / 8 + 1) * sizeof(float2);
  if (inter)
    rope_staged_kernel<T, true><<<grid, NTHREADS, smem, st>>>(a, t);
  else
    rope_staged_kernel<T, false><<<grid, NTHREADS, smem, st>>>(a, t);
}

template <typename T, int VP>
static void launch(const Args& a, const Table& t, bool inter, cudaStream_t st) {
  const int grid = cdiv(a.rows, a.tok);
  const size_t smem = cdiv(a.half, 2) * 16 + (size_t)a.tok * cdiv(a.half, VP) * VP * sizeof(float2) + a.tok * sizeof(int2) + a.half;
  if (inter)
    rope_kernel<T, VP, true><<<grid, NTHREADS, smem, st>>>(a, t);
  else
    rope_kernel<T, VP, false><<<grid, NTHREADS, smem, st>>>(a, t);
}

// {batch, row, head} strides: contiguous when all are zero, otherwise positive
// wherever the dimension has more than one entry (0 where it has not) and, for
// 16-bit types, whole 16-byte units.
static bool strides3(const int64_t in[3], int batch, int seqlen, int heads, int dim, bool vec16, long long out[3]) {
  const bool contiguous = in[0] == 0 && in[1] == 0 && in[2] == 0;
  const int n[3] = {batch, seqlen, heads};
  long long step = dim;
  for (int i = 2; i >= 0; --i) {
    out[i] = n[i] <= 1 ? 0 : contiguous ? step : in[i];
    if (n[i] > 1 && !contiguous && (in[i] <= 0 || in[i] >= (1LL << 36) || (vec16 && in[i] % 8))) return false;
    step *= n[i];
  }
  return true;
}

static int run(const attn_rope_params* p, cudaStream_t st) {
  if (!p) return ATTN_ERR_INVALID_ARG;
  if (p->dtype < ATTN_BF16 || p->dtype > ATTN_FP32) return ATTN_ERR_INVALID_ARG;
  const bool f32 = p->dtype == ATTN_FP32;
  if (p->batch < 0 || p->seqlen < 0 || p->nhead_q < 1 || p->nhead_kv < 0) return ATTN_ERR_INVALID_ARG;
  if ((long long)p->batch * p->seqlen > (1LL << 30) || p->nhead_q > (1 << 20) || p->nhead_kv > (1 << 20))
    return ATTN_ERR_INVALID_ARG;
  if (p->head_dim < 2 || p->head_dim > ATTN_ROPE_MAX_DIM || (!f32 && p->head_dim % 8))
    return ATTN_ERR_UNSUPPORTED_HEADDIM;
  if (p->rot_dim < 2 || p->rot_dim > p->head_dim || p->rot_dim % 2) return ATTN_ERR_INVALID_ARG;
  if (p->n_axes < 1 || p->n_axes > ATTN_ROPE_MAX_AXES) return ATTN_ERR_INVALID_ARG;
  const int half = p->rot_dim / 2;
  if (!p->inv_freq) return ATTN_ERR_INVALID_ARG;
  Table t{};
  for (int i = 0; i < half; ++i) {
    const double f = p->inv_freq[i];
    if (!std::isfinite(f)) return ATTN_ERR_INVALID_ARG;
    t.axis[i] = p->pair_axis ? p->pair_axis[i] : 0;
    if (t.axis[i] >= p->n_axes) return ATTN_ERR_INVALID_ARG;
    // turns per position, whole turns dropped, in units of 2^-64
    double turns = f * 0.15915494309189533577;
    turns -= std::floor(turns);
    const double hi = std::floor(turns * 4294967296.0);            // exact: a shift, then 32 whole bits
    const double lo = (turns * 4294967296.0 - hi) * 4294967296.0;   // exact, below 2^32
    t.step[i] = ((unsigned long long)hi << 32) + (unsigned long long)lo;   // turns = 1.0 wraps to 0
  }
  const bool has_k = p->nhead_kv > 0;
  Args a{};
  long long s[3];
  auto side = [&](const void* in, void* out, const int64_t si[3], const int64_t so[3], int heads, Side* x) {
    const unsigned al = f32 ? 4 : 16;
    if (!in || !out || !aligned_to(in, al) || !aligned_to(out, al)) return false;
    if (!strides3(si, p->batch, p->seqlen, heads, p->head_dim, !f32, s)) return false;
    x->in = in; x->ib = s[0]; x->ir = s[1]; x->ih = s[2];
    if (!strides3(so, p->batch, p->seqlen, heads, p->head_dim, !f32, s)) return false;
    x->out = out; x->ob = s[0]; x->orow = s[1]; x->oh = s[2];
    // in place only element by element
    return in != out || (x->ib == x->ob && x->ir == x->orow && x->ih == x->oh) ||
           (long long)p->batch * p->seqlen == 0;
  };
  const long long rows = (long long)p->batch * p->seqlen;
  if (rows == 0) return ATTN_OK;
  if (!side(p->q, p->q_out, p->stride_q, p->stride_q_out, p->nhead_q, &a.q)) return ATTN_ERR_INVALID_ARG;
  if (has_k && !side(p->k, p->k_out, p->stride_k, p->stride_k_out, p->nhead_kv, &a.k)) return ATTN_ERR_INVALID_ARG;
  if (!p->positions || !aligned_to(p->positions, 4)) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (p->stride_pos[i] < 0 || p->stride_pos[i] >= (1LL << 36)) return ATTN_ERR_INVALID_ARG;
  a.pos = p->positions;
  a.pa = p->stride_pos[0]; a.pb = p->stride_pos[1]; a.pr = p->stride_pos[2];
  a.rows = (int)rows;
  a.seqlen = p->seqlen;
  a.hq = p->nhead_q;
  a.heads = p->nhead_q + p->nhead_kv;
  a.dim = p->head_dim;
  a.half = half;
  a.inverse = p->inverse != 0;
  // Rows of a CTA share the table and the wait for their cosines; fewer where eight
  // would leave SMs idle (16,384 rows of 40 heads of 128: 58.7 us at eight, 60.2 at
  // four, 87 at one; 3,000: 12.9, 11.3 and 15.3; 800: two 5.4, one 6.4; 64: 3.3 at one,
  // 3.7 at two).
  a.tok = a.rows < 600 ? 1 : a.rows < 1500 ? 2 : a.rows < 8000 ? 4 : 8;
  const int vp = f32 ? 4 : 8;
  const bool pairs = p->interleaved ? p->head_dim % (2 * vp) == 0 : half % vp == 0 && p->head_dim % vp == 0;
  bool wide = p->head_dim % vp == 0;   // rows of whole vectors
  if (f32)
    for (const Side* x : {&a.q, &a.k}) {
      if (x == &a.k && !has_k) continue;
      wide = wide && aligned_to(x->in, 16) && aligned_to(x->out, 16) && x->ib % 4 == 0 && x->ir % 4 == 0 &&
             x->ih % 4 == 0 && x->ob % 4 == 0 && x->orow % 4 == 0 && x->oh % 4 == 0;
    }
  const bool inter = p->interleaved != 0;
  if (!wide) launch<float, 1>(a, t, inter, st);   // 16-bit rows always are
  else if (p->dtype == ATTN_BF16) pairs ? launch<__nv_bfloat16, 8>(a, t, inter, st) : launch_staged<__nv_bfloat16>(a, t, inter, st);
  else if (p->dtype == ATTN_FP16) pairs ? launch<__half, 8>(a, t, inter, st) : launch_staged<__half>(a, t, inter, st);
  else pairs ? launch<float, 4>(a, t, inter, st) : launch_staged<float>(a, t, inter, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace rope
}  // namespace attn

extern "C" int attn_rope(const attn_rope_params* p, cudaStream_t stream) { return attn::rope::run(p, stream); }
