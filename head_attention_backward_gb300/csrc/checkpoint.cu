// 8-bit activation checkpoints (attn_checkpoint_save) and their expansion for
// the backward pass (attn_bwd_checkpoint, api.cu).
//
// Whole numbers of 7 bits under a power of two: the step is at most 1/64 of the
// group's largest magnitude, where e4m3 under a power of two would be off by up
// to 1/16 of each value (for a normal distribution four times as much), and a
// number times a power of two is exact in bf16 and fp16, so the backward's
// tensor-core kernel takes the expanded tensors as they are.  Groups of 32
// columns keep a column that stands out from costing the rest of its row its
// steps, for 1/32 of a byte.
//
// Both kernels are bound by memory: 2 bytes read and 1 + 1/32 written per value,
// and the other way round.  Four neighbouring lanes hold a group, 16 bytes of
// 16-bit values each, so every load and store is coalesced and a scale takes two
// shuffles.
#include "ckpt_common.cuh"

namespace attn {
namespace ckpt {

constexpr int THREADS = 256;
constexpr int HELD = 4;                    // pieces of 8 values that a thread holds
constexpr int PER_CTA = THREADS * HELD;

// n / d for n < 2^31: (n + mulhi(n, m)) >> s, the round-up method of Granlund and
// Montgomery, "Division by invariant integers using multiplication" (1994).
struct Div {
  uint32_t d, m, s;
};
static Div make_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {d, (uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Div& d) { return (__umulhi(n, d.m) + n) >> d.s; }

// One tensor in the order of its checkpoint's memory: pieces of 8 columns, then
// three dimensions with the source's element strides.
struct Side {
  const void* x;
  int8_t* n;
  uint8_t* exp;
  uint32_t pieces;                         // of 8 values
  uint32_t first_cta;
  int linear;                              // the source has the same order and no gaps
  Div per_row, d2, d1;                     // pieces of a row and head; sizes of the inner two dimensions
  long long s0, s1, s2;
};
struct Args {
  Side t[4];
};

template <typename T> struct Piece { uint4 w; };           // 8 values
template <> struct Piece<float> { uint4 w, w2; };

template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* at) { return {__ldcs(reinterpret_cast<const uint4*>(at))}; }
template <>
__device__ __forceinline__ Piece<float> load_piece<float>(const float* at) {
  return {__ldcs(reinterpret_cast<const uint4*>(at)), __ldcs(reinterpret_cast<const uint4*>(at) + 1)};
}

// Largest magnitude of a piece, as the bits of an fp32 (they order like the
// magnitudes, infinities and NaN above all).
__device__ __forceinline__ uint32_t amax_bits(const Piece<float>& p) {
  const uint32_t w[8] = {p.w.x, p.w.y, p.w.z, p.w.w, p.w2.x, p.w2.y, p.w2.z, p.w2.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
  return m;
}
template <typename T>
__device__ __forceinline__ uint32_t amax_pair(const Piece<T>& p) {   // in 16-bit halves
  const uint32_t k = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(p.w.x & k, p.w.y & k), __vmaxu2(p.w.z & k, p.w.w & k));
}
__device__ __forceinline__ uint32_t widen(uint32_t half, __nv_bfloat16*) { return half << 16; }
__device__ __forceinline__ uint32_t widen(uint32_t half, __half*) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)half)));
}

// The group's, over its four lanes.
template <typename T>
__device__ __forceinline__ uint32_t group_amax(const Piece<T>& p) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = amax_bits(p);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  } else {
    uint32_t m = amax_pair<T>(p);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return widen(max(m & 0xffffu, m >> 16), (T*)nullptr);
  }
}

// Least e >= CK_EXP_MIN with amax <= 127 * 2^e = 1.984375 * 2^(e + 6).
__device__ __forceinline__ int exponent_of(uint32_t amax) {
  const int e = (int)(amax >> 23) - 127 - 6 + ((amax & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return max(e, CK_EXP_MIN);
}

template <typename T> __device__ __forceinline__ void floats(const Piece<T>& p, float (&f)[8]);
template <> __device__ __forceinline__ void floats<float>(const Piece<float>& p, float (&f)[8]) {
  const uint32_t w[8] = {p.w.x, p.w.y, p.w.z, p.w.w, p.w2.x, p.w2.y, p.w2.z, p.w2.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
template <> __device__ __forceinline__ void floats<__nv_bfloat16>(const Piece<__nv_bfloat16>& p, float (&f)[8]) {
  const uint32_t w[4] = {p.w.x, p.w.y, p.w.z, p.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <> __device__ __forceinline__ void floats<__half>(const Piece<__half>& p, float (&f)[8]) {
  const uint32_t w[4] = {p.w.x, p.w.y, p.w.z, p.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = y.x;
    f[2 * i + 1] = y.y;
  }
}

// Four values over 2^e, to nearest even: the sum with 1.5 * 2^23 leaves the whole
// number in the low byte (x 2^-e is exact or rounds to a number that is 0 anyway).
__device__ __forceinline__ uint32_t pack4(const float* f, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(fmaf(f[i], inv, 12582912.f));
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) save_kernel(const __grid_constant__ Args A) {
  int i = 0;
#pragma unroll
  for (int j = 1; j < 4; ++j) i += blockIdx.x >= A.t[j].first_cta;
  const Side& S = A.t[i];
  const uint32_t v0 = (blockIdx.x - S.first_cta) * PER_CTA + threadIdx.x;
  const T* x = static_cast<const T*>(S.x);
  Piece<T> p[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const uint32_t v = v0 + k * THREADS;
    p[k] = {};
    if (v < S.pieces) {
      long long at = (long long)v * 8;
      if (!S.linear) {
        const uint32_t row = quotient(v, S.per_row), r1 = quotient(row, S.d2), r0 = quotient(r1, S.d1);
        at = (long long)(v - row * S.per_row.d) * 8 + (row - r1 * S.d2.d) * S.s2 + (r1 - r0 * S.d1.d) * S.s1 + r0 * S.s0;
      }
      p[k] = load_piece<T>(x + at);
    }
  }
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const uint32_t v = v0 + k * THREADS;       // groups do not straddle the end: pieces is a multiple of 4
    const uint32_t amax = group_amax<T>(p[k]);
    const bool bad = amax >= 0x7f800000u;
    const int e = exponent_of(amax);
    float f[8];
    floats<T>(p[k], f);
    const float inv = __int_as_float((127 - e) << 23);
    const uint2 n = bad ? make_uint2(0u, 0u) : make_uint2(pack4(f, inv), pack4(f + 4, inv));
    if (v < S.pieces) {
      __stcs(reinterpret_cast<uint2*>(S.n) + v, n);
      if ((v & 3) == 0) S.exp[v >> 2] = (uint8_t)(bad ? CK_NAN : e + CK_EXP_BIAS);
    }
  }
}

// ------------------------------------------------------------- expansion

struct Wide {
  const int8_t* n;
  const uint8_t* exp;
  void* y;
  uint32_t pieces, first_cta;
};
struct ExpandArgs {
  Wide t[4];
};

template <typename T>
__device__ __forceinline__ uint32_t pack2t(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2t<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2t<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Every value is exact in T if the checkpoint's tensors were of that type.  In fp16 those
// of a wider type's are limited to 65504 and rounded below 2^-14.
template <typename T>
__global__ void __launch_bounds__(THREADS) expand_kernel(const __grid_constant__ ExpandArgs A) {
  int i = 0;
#pragma unroll
  for (int j = 1; j < 4; ++j) i += blockIdx.x >= A.t[j].first_cta;
  const Wide& S = A.t[i];
  const uint32_t v0 = (blockIdx.x - S.first_cta) * PER_CTA + threadIdx.x;
  uint2 n[HELD];
  uint32_t e[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const uint32_t v = v0 + k * THREADS;
    n[k] = make_uint2(0u, 0u);
    e[k] = 0;
    if (v < S.pieces) {
      n[k] = __ldcs(reinterpret_cast<const uint2*>(S.n) + v);
      e[k] = __ldg(S.exp + (v >> 2));
    }
  }
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const uint32_t v = v0 + k * THREADS;
    if (v >= S.pieces) break;
    float f[8];
    ck_values8<T>(n[k], ck_scale(e[k]), f);
    uint4* y = static_cast<uint4*>(S.y);
    if constexpr (sizeof(T) == 4) {
      y[2 * (size_t)v] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      y[2 * (size_t)v + 1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    } else {
      y[v] = make_uint4(pack2t<T>(f[0], f[1]), pack2t<T>(f[2], f[3]), pack2t<T>(f[4], f[5]), pack2t<T>(f[6], f[7]));
    }
  }
  // complete only after the kernel that it ran beside
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// -------------------------------------------------------------------- host

// Most values of a tensor: pieces and their quotients stay below 2^31.
constexpr long long MAX_VALUES = 1LL << 33;

static int save(const attn_checkpoint_params* p, cudaStream_t st) {
  if (!p || p->dtype < ATTN_BF16 || p->dtype > ATTN_FP32) return ATTN_ERR_INVALID_ARG;
  if (p->batch < 1 || p->nhead_q < 1 || p->nhead_kv < 1 || p->seqlen_q < 0 || p->seqlen_k < 0) return ATTN_ERR_INVALID_ARG;
  if (!ck_headdim(p->d_qk) || !ck_headdim(p->d_v)) return ATTN_ERR_UNSUPPORTED_HEADDIM;
  const attn_checkpoint& c = p->ckpt;
  const void* from[4] = {p->q, p->k, p->v, p->o};
  const int64_t* in[4] = {p->stride_q, p->stride_k, p->stride_v, p->stride_o};
  int8_t* to[4] = {c.q, c.k, c.v, c.o};
  uint8_t* exps[4] = {c.q_exp, c.k_exp, c.v_exp, c.o_exp};
  const int64_t* out[4] = {c.stride_q, c.stride_k, c.stride_v, c.stride_o};
  Args a{};
  uint32_t ctas = 0;
  for (int i = 0; i < 4; ++i) {
    const bool q_side = i == 0 || i == 3;
    const long long size[3] = {p->batch, q_side ? p->seqlen_q : p->seqlen_k, q_side ? p->nhead_q : p->nhead_kv};
    const int d = i < 2 ? p->d_qk : p->d_v;
    Side& t = a.t[i];
    t.first_cta = ctas;
    if (size[0] * size[1] > (1LL << 30) || size[0] * size[1] * size[2] > MAX_VALUES / d) return ATTN_ERR_INVALID_ARG;
    const long long rows = size[0] * size[1] * size[2];
    t.pieces = (uint32_t)(rows * (d / 8));
    int order[3];
    long long own[3];
    if (!ck_dense(out[i], size, d, own, order)) return ATTN_ERR_INVALID_ARG;
    if (rows == 0) continue;
    if (!from[i] || !to[i] || !exps[i] || !ck_aligned(from[i]) || !ck_aligned(to[i])) return ATTN_ERR_INVALID_ARG;
    long long src[3] = {size[1] * size[2] * d, size[2] * d, d};
    if (in[i][0] != 0 || in[i][1] != 0 || in[i][2] != 0) {
      for (int k = 0; k < 3; ++k) {
        if (size[k] > 1 && (in[i][k] <= 0 || in[i][k] >= (1LL << 36) || in[i][k] % 8 != 0)) return ATTN_ERR_INVALID_ARG;
        src[k] = size[k] > 1 ? in[i][k] : 0;
      }
    }
    t.x = from[i];
    t.n = to[i];
    t.exp = exps[i];
    t.linear = 1;
    for (int k = 0; k < 3; ++k) t.linear &= size[k] == 1 || src[k] == own[k];
    t.per_row = make_div(d / 8);
    t.d2 = make_div((uint32_t)size[order[2]]);
    t.d1 = make_div((uint32_t)size[order[1]]);
    t.s0 = src[order[0]];
    t.s1 = src[order[1]];
    t.s2 = src[order[2]];
    ctas += cdiv_ll(t.pieces, PER_CTA);
  }
  if (ctas == 0) return ATTN_OK;
  if (p->dtype == ATTN_BF16) save_kernel<__nv_bfloat16><<<ctas, THREADS, 0, st>>>(a);
  else if (p->dtype == ATTN_FP16) save_kernel<__half><<<ctas, THREADS, 0, st>>>(a);
  else save_kernel<float><<<ctas, THREADS, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace ckpt

bool ck_headdim(int d) { return d >= 32 && d <= 256 && d % 32 == 0; }

// The tensor's strides (the contiguous ones for three zeros) if it has no gaps, and
// its dimensions from the outermost to the innermost.  A dimension of one entry
// carries any stride and gets that of the place it is sorted to.
bool ck_dense(const int64_t in[3], const long long size[3], int d, long long own[3], int order[3]) {
  const bool zero = in[0] == 0 && in[1] == 0 && in[2] == 0;
  for (int k = 0; k < 3; ++k) order[k] = k;
  if (!zero) {
    // an insertion sort by stride, descending; dimensions of one entry stay where they are
    for (int k = 1; k < 3; ++k)
      for (int j = k; j > 0; --j) {
        const int a = order[j - 1], b = order[j];
        if (size[a] > 1 && size[b] > 1 && in[a] >= in[b]) break;
        if (size[b] <= 1) break;
        order[j - 1] = b;
        order[j] = a;
      }
  }
  long long next = d;
  for (int k = 2; k >= 0; --k) {
    const int x = order[k];
    if (!zero && size[x] > 1 && in[x] != next) return false;
    own[x] = next;
    next *= size[x] > 0 ? size[x] : 1;
  }
  return true;
}

bool launch_ck_expand(const CkExpand& x, bool beside, cudaStream_t st) {
  ckpt::ExpandArgs a{};
  uint32_t ctas = 0;
  for (int i = 0; i < 4; ++i) {
    a.t[i] = {x.n[i], x.exp[i], x.y[i], (uint32_t)(x.values[i] / 8), ctas};
    ctas += (uint32_t)cdiv_ll(x.values[i] / 8, ckpt::PER_CTA);
  }
  if (ctas == 0) return true;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(ckpt::THREADS);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = beside ? 1 : 0;
  const cudaError_t e = x.dtype == ATTN_BF16   ? cudaLaunchKernelEx(&cfg, ckpt::expand_kernel<__nv_bfloat16>, a)
                        : x.dtype == ATTN_FP16 ? cudaLaunchKernelEx(&cfg, ckpt::expand_kernel<__half>, a)
                                               : cudaLaunchKernelEx(&cfg, ckpt::expand_kernel<float>, a);
  return e == cudaSuccess;
}

}  // namespace attn

extern "C" int attn_checkpoint_save(const attn_checkpoint_params* p, cudaStream_t stream) {
  return attn::ckpt::save(p, stream);
}
