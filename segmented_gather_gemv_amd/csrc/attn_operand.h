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

// Eight codes with those that are not finite (e4m3: 0x7f and 0xff) replaced by finite ones.
template <int FMT>
__device__ __forceinline__ u32x2_t finite_codes(u32x2_t w) {
  if constexpr (FMT == SGMV_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] &= ~((((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7);
  }
  return w;
}

// Bit 15 of each bf16 of a word that is not finite: its exponent is all ones, so that one more carries.
__device__ __forceinline__ uint32_t nonfinite_flags(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// Both bytes of each half whose bit 15 is set.
__device__ __forceinline__ uint32_t flag_mask(uint32_t f) { return (f - (f >> 15)) | f; }

// bf16 or fp32 elements only: 8-bit codes are finite.
template <int BYTES>
__device__ __forceinline__ bool has_nonfinite(u32x4_t w) {
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
    if constexpr (BYTES == 2) w[i] &= ~flag_mask(nonfinite_flags(w[i]));
    else if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] = 0u;
  }
  return w;
}

}  // namespace sgmv
