// The 8-bit activation checkpoint's numbers: whole numbers of -127 .. 127 times a
// power of two per group of 32 columns.
#pragma once

#include "common.cuh"

namespace attn {

constexpr int CK_EXP_BIAS = 127;
constexpr int CK_EXP_MIN = -126;    // scales stay normal fp32 numbers
constexpr int CK_NAN = 255;         // exponent byte of a group with an infinity or a NaN

// An 8-bit checkpoint's o in place of o (its strides are the problem's so_), or nulls.
struct CkO {
  const int8_t* n;
  const uint8_t* exp;
};
// What a backward pass expands of a checkpoint: q, k, v (fp32: and o).
struct CkExpand {
  CkO o;
  int dtype;
  const int8_t* n[4];
  const uint8_t* exp[4];
  void* y[4];
  long long values[4];
};

// checkpoint.cu: supported head dims; the strides and dimension order (outermost
// first) of a tensor without gaps; expansion of up to four tensors.
bool ck_headdim(int d);
bool ck_dense(const int64_t in[3], const long long size[3], int d, long long own[3], int order[3]);
// beside: it may run beside the preprocess kernel launched just before it.
bool launch_ck_expand(const CkExpand& x, bool beside, cudaStream_t st);

inline bool ck_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 2^(byte - 127), NaN for the byte that marks a group.
__device__ __forceinline__ float ck_scale(uint32_t byte) {
  return byte == CK_NAN ? __int_as_float(0x7fffffff) : __uint_as_float(byte << 23);
}

// Four whole numbers as fp32: a byte b in the low mantissa bits of 2^23 reads
// 2^23 + b, and with its sign bit flipped b is the number + 128.
__device__ __forceinline__ void ck_unpack4(uint32_t x, float (&y)[4]) {
  x ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440 + i)) - 8388736.f;
}

// Values of a type past its largest finite one are that (a rounded up fp16 or bf16
// amax); NaN stays.
template <typename T> __device__ __forceinline__ float ck_limit(float x) { return x; }
template <> __device__ __forceinline__ float ck_limit<__half>(float x) {
  return fabsf(x) > 65504.f ? copysignf(65504.f, x) : x;
}
template <> __device__ __forceinline__ float ck_limit<__nv_bfloat16>(float x) {
  return fabsf(x) > 3.3895313892515355e38f ? copysignf(3.3895313892515355e38f, x) : x;
}
template <> __device__ __forceinline__ float ck_limit<float>(float x) {
  return fabsf(x) > 3.4028234663852886e38f ? copysignf(3.4028234663852886e38f, x) : x;
}

// Eight numbers of one group as the values that they stand for.
template <typename T>
__device__ __forceinline__ void ck_values8(uint2 n, float scale, float (&y)[8]) {
  float a[4], b[4];
  ck_unpack4(n.x, a);
  ck_unpack4(n.y, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = ck_limit<T>(a[i] * scale);
    y[4 + i] = ck_limit<T>(b[i] * scale);
  }
}

}  // namespace attn
