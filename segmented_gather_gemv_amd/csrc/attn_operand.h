// Operands of V as stored: which tokens to keep, and values that are not finite.
#pragma once

#include "attn.h"

namespace sgmv {

// The bits of a word of two bf16 whose flag is set.
__device__ __forceinline__ uint32_t keep_pair(uint32_t w, uint32_t two) {
  return w & ((two & 1 ? 0x0000ffffu : 0u) | (two & 2 ? 0xffff0000u : 0u));
}

// Keep the elements of a 16-byte piece whose bit of `keep` is set (bit i: element i), zero the others.
template <int BYTES>
__device__ __forceinline__ u32x4_t keep_elements(u32x4_t w, uint32_t keep) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BYTES == 1) {
      const uint32_t m = keep >> (4 * i);
      w[i] &= (m & 1 ? 0xffu : 0u) | (m & 2 ? 0xff00u : 0u) | (m & 4 ? 0xff0000u : 0u) | (m & 8 ? 0xff000000u : 0u);
    } else if constexpr (BYTES == 2) {
      w[i] = keep_pair(w[i], keep >> (2 * i));
    } else {
      w[i] = keep >> i & 1 ? w[i] : 0u;
    }
  }
  return w;
}

// The places (16 bits, in V's order) of a group's first n tokens.
__device__ __forceinline__ uint32_t places_below(int n) {
  const uint32_t t = (1u << n) - 1u;  // tokens 4-7 and 8-11 change places
  return (t & 0xf00fu) | (t & 0x00f0u) << 4 | (t & 0x0f00u) >> 4;
}

// The places of the group of tokens [g0, g0 + 16) that a row at position pos sees.
__device__ __forceinline__ uint32_t places_seen(const AttnArgs& A, int pos, int g0) {
  const int n = max(pos - g0 + 1, 0);
  return places_below(min(n, 16)) & ~(A.window ? places_below(min(max(n - A.window, 0), 16)) : 0u);
}

// The places of a group whose scale (of 16 tokens in order) is not finite.
__device__ __forceinline__ uint32_t places_of_nan(const float* scale) {
  uint32_t odd = 0;
#pragma unroll
  for (int t = 0; t < KV_GROUP; ++t)
    if (!(fabsf(scale[t]) < INFINITY)) odd |= places_below(t + 1) & ~places_below(t);
  return odd;
}

// Bit 7 of each byte of a word that is an e4m3 code of NaN (0x7f, 0xff).
__device__ __forceinline__ uint32_t nan_code_flags(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Not 0 if a code of a 16-byte piece is NaN.
__device__ __forceinline__ uint32_t nan_code_any(u32x4_t w) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
  return any & 0x80808080u;
}

// Bit 7 of each byte (token) of a 16-byte piece of codes whose bit of `places` is set.
__device__ __forceinline__ u32x4_t place_flags(uint32_t places) {
  u32x4_t f;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // bit k of four to bit 8 k
    f[i] = ((places >> (4 * i) & 15u) * 0x204081u & 0x01010101u) << 7;
  return f;
}

// Whether one of a piece's codes is NaN, among those with a flag.
__device__ __forceinline__ bool nan_among(u32x4_t w, u32x4_t flags) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= nan_code_flags(w[i]) & flags[i];
  return any != 0u;
}

// Bit 15 of each bf16 of a word that is not finite: its exponent is all ones, so that one more carries.
__device__ __forceinline__ uint32_t nonfinite_flags(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// Both bytes of each half whose bit 15 is set.
__device__ __forceinline__ uint32_t flag_mask(uint32_t f) { return (f - (f >> 15)) | f; }

// One byte: e4m3 codes (int8 has none of NaN).
template <int BYTES>
__device__ __forceinline__ bool has_nonfinite(u32x4_t w) {
  if constexpr (BYTES == 1) return nan_code_any(w) != 0u;
  if constexpr (BYTES == 2)
    return (nonfinite_flags(w.x) | nonfinite_flags(w.y) | nonfinite_flags(w.z) | nonfinite_flags(w.w)) != 0u;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= (w[i] & 0x7f800000u) == 0x7f800000u;
  return any;
}

template <int BYTES>
__device__ __forceinline__ u32x4_t drop_nonfinite(u32x4_t w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BYTES == 1) w[i] &= ~(nan_code_flags(w[i]) >> 7);
    else if constexpr (BYTES == 2) w[i] &= ~flag_mask(nonfinite_flags(w[i]));
    else if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] = 0u;
  }
  return w;
}

}  // namespace sgmv
