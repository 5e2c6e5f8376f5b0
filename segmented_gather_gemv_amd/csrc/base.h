// Product with a base weight held in 4 bits: arguments and the operands that both kernels share.
//
// A block of 16 n and 128 k is 1 KB, 16 bytes of each lane; its word j is the right operand of the 16x16x32
// product over k = 32 j .. 32 j + 31 once converted: lane (n = lane % 16, quad = lane / 16) holds k = 8 quad .. + 7 of
// column n. The left operand is 16 rows of x; lane (n, quad) gets rows 4 quad .. 4 quad + 3 of column n, so that a
// group's scale and zero point are one value of the lane.
//   I4    c is an e4m3 code as it stands (a number below 16 in the low bits of a byte is c 2^-9), so that two codes
//         become two exact bf16 by one instruction: y += s (sum c x - z sum x), with sum x from a product by ones.
//         (Both sums are of one sign where x is, and cancel: roundings count against s (c + z) |x|.)
//   E2M1  the scale is a power of two, which the conversion applies: the operand is the weight itself, exact.
// fp32 rows are split into three bf16 (24 bits).
#pragma once

#include <type_traits>

#include "common.h"

namespace sgmv {

constexpr int BASE_K = 128;  // k of a block
constexpr int BASE_N = 16;   // n

struct BaseArgs {
  const void* codes;
  const void* scale;
  const uint8_t* zero;
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int32_t T, N, K;
  int32_t blocks;      // of 128 k
  int32_t scale_rows;  // [16][s] rows of scales of 16 n
  int32_t per_group;   // blocks of a group (1 for short ones)
  // tiled kernel
  char* rows;          // x in blocks of a tile's rows and 128 k, with their sums (base_tiled.hip)
  int32_t y_vec;       // rows of y may be written 16 bytes at a time
  int32_t splits, split_blocks;  // ranges of K, and their blocks
  float* parts;        // their sums, where there are several
};

struct BasePackArgs {
  const uint8_t* codes;
  int64_t ldc;
  const void* scale;
  const uint8_t* zero;
  void *codes_out, *scale_out;
  uint8_t* zero_out;
  int32_t N, K, groups, blocks, scale_rows, s, e2m1, scale_bytes;
};

// Rows and columns of a workgroup of the tiled kernel.
constexpr int TILE_T = 64;
constexpr int TILE_N = 256;

hipError_t launch_base_tiled(const BaseArgs& A, int format, int dtype, int s, hipStream_t stream);
hipError_t launch_base_pack(const BasePackArgs& A, hipStream_t stream);
hipError_t launch_base_direct_i4(const BaseArgs& A, int s, hipStream_t stream);
hipError_t launch_base_direct_i4z(const BaseArgs& A, int s, hipStream_t stream);
hipError_t launch_base_direct_e2m1(const BaseArgs& A, hipStream_t stream);
hipError_t launch_base_direct_f32(const BaseArgs& A, int format, int s, hipStream_t stream);

// Eight I4 codes as bf16.
__device__ __forceinline__ u32x4_t base_codes(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 512.f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 512.f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 512.f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 512.f, true))};
}

// Eight E2M1 codes times a power of two, as bf16.
__device__ __forceinline__ u32x4_t base_floats(uint32_t w, float scale) {
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
}

// The scales of one row of 16 n, kept as they were loaded (what converts them waits for them); E2M1's as what the
// conversion takes.
template <bool E2M1, bool F32, int S>
struct BaseScale {
  static constexpr int BITS = E2M1 ? 8 : F32 ? 32 : 16, WORDS = (S * BITS + 31) / 32;
  uint32_t w[WORDS];
  static __device__ __forceinline__ BaseScale load(const void* p, int64_t row, int n) {
    BaseScale r;
    const char* q = static_cast<const char*>(p) + (row * BASE_N + n) * (S * BITS / 8);
    if constexpr (S * BITS == 16) {
      r.w[0] = *reinterpret_cast<const uint16_t*>(q);
    } else if constexpr (WORDS == 2) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(q);
      r.w[0] = v.x;
      r.w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(q)[i];
    }
    return r;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (E2M1) return __uint_as_float((w[0] >> (8 * i) & 255u) << 23);
    else if constexpr (F32) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// Zero points of one row of 16 n (8 where there are none).
template <bool ZERO, int S>
struct BaseZero {
  uint32_t w;
  static __device__ __forceinline__ BaseZero load(const uint8_t* p, int64_t row, int n) {
    BaseZero r{0u};
    if constexpr (ZERO) {
      const uint8_t* q = p + (row * BASE_N + n) * S;
      if constexpr (S == 4) r.w = *reinterpret_cast<const uint32_t*>(q);
      else if constexpr (S == 2) r.w = *reinterpret_cast<const uint16_t*>(q);
      else r.w = *q;
    }
    return r;
  }
  __device__ __forceinline__ float get(int i) const { return ZERO ? (float)(w >> (8 * i) & 255u) : 8.f; }
};

// Keeps a wave's LDS accesses before it in front of those behind it, for values that its lanes pass to each other there.
// (The hardware carries out a wave's LDS accesses in order: this is for the compiler, and makes no instruction.)
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// 16 bytes of a row, wherever it starts.
template <bool F32>
__device__ __forceinline__ u32x4_t load_row(const char* p) {
  typedef u32x4_t by_4_t __attribute__((aligned(4)));
  typedef u32x4_t by_2_t __attribute__((aligned(2)));
  return *reinterpret_cast<const std::conditional_t<F32, by_4_t, by_2_t>*>(p);
}

// The same, of a piece that ends n values on, zeros behind them.
template <bool F32>
__device__ __forceinline__ u32x4_t load_rest(const char* p, int n) {
  u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 8); ++i)
    if (i < n) {
      if constexpr (F32) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else v[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
  return v;
}

// fp32 values as three bf16 each that add up to them: their leading 8 bits, the next 8, the last (numbers below
// 2^-110 lose bits that bf16 does not hold).
__device__ __forceinline__ void split3(const u32x4_t (&x)[2], bf16x8_t (&p)[3]) {
  u32x4_t w[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = x[i / 2][2 * (i % 2)], b = x[i / 2][2 * (i % 2) + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      w[k][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      a = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & 0xffff0000u));
      b = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & 0xffff0000u));
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) p[k] = as_bf16x8(w[k]);
}

}  // namespace sgmv
