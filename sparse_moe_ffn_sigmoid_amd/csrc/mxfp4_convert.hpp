// MXFP4 encoding of values in registers.
#pragma once

#include "common.hpp"

namespace moe {
namespace mx {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// Element types by moe_dtype
template <int DT>
struct Elem;
template <>
struct Elem<MOE_F32> {
  typedef float type;
  static __device__ __forceinline__ float f32(float v) { return v; }
};
template <>
struct Elem<MOE_BF16> {
  typedef bf16_t type;
  static __device__ __forceinline__ float f32(bf16_t v) { return bf16_to_f32(v); }
};
template <>
struct Elem<MOE_F16> {
  typedef _Float16 type;
  static __device__ __forceinline__ float f32(_Float16 v) { return static_cast<float>(v); }
};

// Scale byte of a block from the largest magnitude's fp32 bits (the largest
// bit pattern is the largest magnitude, and any infinity or NaN is above all
// finite ones).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = static_cast<int>(amax_bits >> 23);
  return e > 2 ? e - 2 : 0;  // amax < 2^-124 (zero and subnormals among it): the exponent clamps
}

__device__ __forceinline__ float scale_value(uint32_t sb) {
  return __uint_as_float(sb ? sb << 23 : 0x00400000u);  // 2^(sb - 127), a subnormal at 0
}

// E2M1 code of q = v / 2^X (exact: a scaling by a power of two)
__device__ __forceinline__ uint32_t e2m1(float q) {
  const float a = fabsf(q);
  const uint32_t c = a <= 0.25f ? 0u : a < 0.75f ? 1u : a <= 1.25f ? 2u : a < 1.75f ? 3u
                   : a <= 2.5f ? 4u : a < 3.5f ? 5u : a <= 5.0f ? 6u : 7u;
  return c | ((__float_as_uint(q) >> 31) << 3);
}

// 8 values -> 8 codes in a word, element 0 in the low nibble.  The hardware
// conversion divides by the scale and rounds to nearest even; blocks at the
// bottom of the exponent range, whose elements or scale are subnormal, are
// compared with the halfway points instead.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t sb) {
  if (sb == 255u) return 0u;
  uint32_t w = 0;
  if (sb < 4u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= e2m1(ldexpf(v[i], 127 - static_cast<int>(sb))) << (4 * i);
    return w;
  }
#if defined(__HIP_DEVICE_COMPILE__)
  const float sc = scale_value(sb);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
#endif
  return w;
}

// The bits of 8 elements of a row, zeros behind `left` of them; one or two
// 16-byte loads where the row allows it.
template <int DT>
struct Raw8 {
  typedef typename Elem<DT>::type E;
  __attribute__((aligned(16))) uint32_t w[2 * sizeof(E)];

  __device__ __forceinline__ void load(const E* p, int64_t left, bool vec) {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    if (vec && left >= 8) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(E)) / 2; ++i)
        *reinterpret_cast<u32x4_t*>(w + 4 * i) = reinterpret_cast<const u32x4_t*>(p)[i];
    } else {
      E e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < left ? p[i] : E(0);
      __builtin_memcpy(w, e, sizeof(w));
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    E e[8];
    __builtin_memcpy(e, w, sizeof(w));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<DT>::f32(e[i]);
  }
};

template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* p, int64_t left, bool vec,
                                      float (&v)[8]) {
  Raw8<DT> raw;
  raw.load(p, left, vec);
  raw.values(v);
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// max over the four lanes of a block of a row
__device__ __forceinline__ uint32_t max4(uint32_t m) {
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1, 4)));
  return max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2, 4)));
}

}  // namespace mx
}  // namespace moe
