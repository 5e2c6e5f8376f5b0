// Codes of a row's values in the 8-bit formats: with F = 448 (e4m3) or 127 (int8),
//   amax = max |x|,  scale = amax / F,  code = round(x * F / amax) to the format, ties to even
// (kv_cache.hip says how the code is that of the exact quotient).
#pragma once

#include "kv_common.h"

namespace sgmv {

// fp32 nearest to d, rounded to odd: a later rounding to fewer bits then equals a single one.
__device__ __forceinline__ float to_odd(double d) {
  const float f = __double2float_rz(d);
  return (double)f == d ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// What quantising a row needs: its maximum; a power of two that keeps the parts of a quotient in range, and F
// over the maximum so scaled (0: codes 0); its scale.
struct RowScale {
  float amax, s, inv, scale;
};

// top: bits of the row's maximum of |x| (as integers they order as the values do, infinity and NaN last)
template <int FMT>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
  if (top == 0u || top >= 0x7f800000u) return {0.f, 1.f, 0.f, top ? __uint_as_float(0x7fc00000u) : 0.f};
  const float amax = __uint_as_float(top), s = amax > 0x1p100f ? 0x1p-32f : amax < 0x1p-90f ? 0x1p64f : 1.f;
  return {amax, s, F / (amax * s), amax / F};
}

// Four values rounded to codes. int8: the low bits of 1.5 * 2^23 + q are those of q rounded.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float (&q)[4]) {
  if constexpr (FMT == SGMV_KV_E4M3) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  } else {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 0x1.8p23f);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
  }
}

// Codes of four values of a row.
template <int FMT, class T>
__device__ __forceinline__ uint32_t quantise4(const float (&x)[4], const RowScale& S) {
  constexpr float F = FMT == SGMV_KV_E4M3 ? 448.f : 127.f;
  uint32_t w;
  float q[4];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __uint_as_float((__float_as_uint(x[i] * S.s * S.inv) + 16u) & ~31u);
    w = encode4<FMT>(q);
  } else {
    float hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = x[i] * S.s * S.inv;
      q[i] = y * (1.f - 0x1p-22f);
      hi[i] = y * (1.f + 0x1p-22f);
    }
    w = encode4<FMT>(q);
    if (__any(w != encode4<FMT>(hi))) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = to_odd((double)x[i] * (double)F / (double)S.amax);
      w = encode4<FMT>(q);
    }
  }
  return S.inv == 0.f ? 0u : w;
}

}  // namespace sgmv
